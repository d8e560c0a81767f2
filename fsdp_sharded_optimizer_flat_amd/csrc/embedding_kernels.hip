// embedding_kernels.hip -- embedding lookup with scaling, and the table's gradient
// by sorted tokens.
//
// Gradient: tokens are sorted (stable: equal tokens keep the order of their rows),
// each wave adds up the rows of a segment of the sorted list over a slab of
// columns, and what belongs to one token alone within a segment is written at
// once.  A token whose rows lie in several segments leaves one partial sum per
// segment; they are joined in order.  So the work is even whatever the tokens
// are (one token named by every row too), no atomics decide an order, and each
// row of the gradient is rounded once.
//
// The lookup is bound by memory (20001 rows of 1280, binary32 to bf16: 154 MB in 17.7
// us of kernel).  So is the gradient of a whole table, by its clearing: 16384 rows of 4096 into
// 128256 of bf16 take 155 us to clear 1.05 GB (6.8 TB/s, with the sorting behind it),
// 9.3 to put the sorted chunks together, 68 for the sums (which wait for the cleared
// lines to be written back: the whole call takes 67 where the gradient is added to what
// is there) and 10 for the runs of several segments.  Small ones are bound by their
// launches' latencies: 1024 rows of 1280 into 50304 take 18 us to clear, 6.6 and 4.1.
#include <algorithm>
#include <type_traits>

#include "embedding.h"
#include "octs.h"

namespace zero {
namespace {

using namespace dev;

// One thread per eight elements of out.
template <typename T, typename O>
__global__ __launch_bounds__(kBlock) void embedding_kernel(EmbeddingArgs a, int64_t row0, uint32_t octs,
                                                           uint32_t total)
{
    const uint32_t i = blockIdx.x * kBlock + threadIdx.x;
    if (i >= total)
        return;
    const int64_t r = row0 + i / octs;
    const int c = (int)(i % octs) * kOct, n = min(a.hidden - c, kOct);
    const int64_t t = a.tokens[r];
    float x[kOct];
    if (t >= 0 && t < a.vocab) {
        load_n(static_cast<const T *>(a.table) + t * a.stride + c, n, x);
#pragma unroll
        for (int k = 0; k < kOct; ++k)
            x[k] *= a.scale;
    } else {
#pragma unroll
        for (int k = 0; k < kOct; ++k)
            x[k] = t < 0 ? 0.0f : __builtin_nanf("");
    }
    store_n(static_cast<O *>(a.out) + r * a.out_stride + c, n, x);
}

// -- sorting tokens ----------------------------------------------------------------------

constexpr int kSortBlock = 1024, kSortWaves = kSortBlock / kWave;
constexpr int kDigit = 7, kDigits = 1 << kDigit;   // three passes hold ZERO_MAX_VOCAB and one more
constexpr int kPerThread = kMaxSortChunk / kSortBlock;
static_assert(ZERO_MAX_VOCAB < 1 << (3 * kDigit), "a token and the mark of no token fit three digits");

struct SortShared {
    uint32_t key[kMaxSortChunk];
    uint16_t at[kMaxSortChunk];
    uint32_t count[kDigits * kSortWaves];   // [digit][wave]
    uint32_t wave_sum[kSortWaves];
};

// Sorts n <= kMaxSortChunk tokens by value, stable, by digits from the lowest: a
// wave ranks 64 neighbours by a digit with one ballot per bit, a scan over (digit,
// wave) places them.
__device__ void sort_chunk(const EmbeddingGradArgs &a, int first, int n, SortShared &sh)
{
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int rounds = (n + kSortBlock - 1) / kSortBlock;
    const int wave0 = wave * rounds * kWave;   // each wave's own consecutive positions
    uint32_t key[kPerThread];
    uint16_t at[kPerThread], rank[kPerThread];
    for (int i = 0; i < rounds; ++i) {
        const int p = wave0 + i * kWave + lane;
        uint32_t k = ~0u;                       // behind the last token
        if (p < n) {
            const int64_t t = a.tokens[first + p];
            k = t >= 0 && t < a.vocab ? (uint32_t)t : (uint32_t)a.vocab;
        }
        sh.key[p] = k;
        sh.at[p] = (uint16_t)p;
    }
    const int passes = (32 - __builtin_clz((unsigned)a.vocab) + kDigit - 1) / kDigit;
    for (int pass = 0; pass < passes; ++pass) {
        for (int i = tid; i < kDigits * kSortWaves; i += kSortBlock)
            sh.count[i] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            if (i >= rounds)
                break;
            const int p = wave0 + i * kWave + lane;
            key[i] = sh.key[p];
            at[i] = sh.at[p];
            const uint32_t d = key[i] >> (pass * kDigit) & (kDigits - 1);
            uint64_t same = ~0ull;
#pragma unroll
            for (int b = 0; b < kDigit; ++b) {
                const uint64_t one = __ballot(d >> b & 1);
                same &= d >> b & 1 ? one : ~one;
            }
            const int before = __popcll(same & ((1ull << lane) - 1));
            volatile uint32_t *c = &sh.count[d * kSortWaves + wave];
            const uint32_t seen = *c;
            __builtin_amdgcn_wave_barrier();
            if (before == 0)
                *c = seen + (uint32_t)__popcll(same);
            __builtin_amdgcn_wave_barrier();
            rank[i] = (uint16_t)(seen + before);
        }
        __syncthreads();
        // exclusive scan of the counts, two to a thread
        const uint32_t c0 = sh.count[2 * tid], c1 = sh.count[2 * tid + 1];
        uint32_t sum = c0 + c1;
#pragma unroll
        for (int off = 1; off < kWave; off *= 2) {
            const uint32_t o = __shfl_up(sum, off, kWave);
            sum += lane >= off ? o : 0;
        }
        if (lane == kWave - 1)
            sh.wave_sum[wave] = sum;
        __syncthreads();
        uint32_t base = sum - c0 - c1;
        for (int w = 0; w < wave; ++w)
            base += sh.wave_sum[w];
        sh.count[2 * tid] = base;
        sh.count[2 * tid + 1] = base + c0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            if (i >= rounds)
                break;
            const uint32_t d = key[i] >> (pass * kDigit) & (kDigits - 1);
            const uint32_t p = sh.count[d * kSortWaves + wave] + rank[i];
            sh.key[p] = key[i];
            sh.at[p] = at[i];
        }
        __syncthreads();
    }
    for (int p = tid; p < n; p += kSortBlock) {
        a.chunk_key[first + p] = sh.key[p];
        a.chunk_row[first + p] = (uint32_t)(first + sh.at[p]);
    }
    if (a.samples && tid < kSamples) {
        const int p = (tid + 1) * (a.chunk / kSamples) - 1;
        a.samples[first / a.chunk * kSamples + tid] = p < n ? sh.key[p] : ~0u;
    }
}

// Elements of the gradient that a workgroup clears.
constexpr int kClearOcts = 8 * kSortBlock;

// The first `chunks` workgroups sort a chunk each, the others clear a span of the
// gradient each meanwhile (one after another in memory: 155 us for 128256 x 4096 bf16;
// with a share of the whole to each of as many as fit the device at once, the last of
// them started when the sorting was over, 15 us more).
template <typename T>
__global__ __launch_bounds__(kSortBlock) void sort_and_clear_kernel(EmbeddingGradArgs a, int chunks)
{
    __shared__ SortShared sh;
    if ((int)blockIdx.x < chunks) {
        const int first = blockIdx.x * a.chunk;
        sort_chunk(a, first, min(a.rows - first, a.chunk), sh);
        return;
    }
    const int64_t span = (int64_t)(blockIdx.x - chunks) * kClearOcts;
    T *p = static_cast<T *>(a.d_table);
    if (a.table_stride == a.hidden) {
        // one run of elements, by 16 bytes; its ends off them go one by one
        constexpr int W = 16 / sizeof(T), Per = kOct / W;
        const int64_t n = (int64_t)a.vocab * a.hidden;
        const int64_t head = min((int64_t)((16 - reinterpret_cast<uintptr_t>(p) % 16) % 16 / sizeof(T)), n);
        const int64_t body = (n - head) / W, first = span * Per, last = min(body, first + kClearOcts * Per);
        u32x4 *q = reinterpret_cast<u32x4 *>(p + head);
        for (int64_t i = first + threadIdx.x; i < last; i += kSortBlock)
            q[i] = u32x4{0, 0, 0, 0};
        const int rest = (int)(n - body * W);   // before and behind the body: fewer than 2 W
        if (span == 0 && (int)threadIdx.x < rest)
            p[(int)threadIdx.x < head ? (int64_t)threadIdx.x : (int64_t)threadIdx.x + body * W] = T(0);
        return;
    }
    const int64_t octs = (a.hidden + kOct - 1) / kOct, total = min(octs * a.vocab, span + kClearOcts);
    const float none[kOct] = {};
    for (int64_t i = span + threadIdx.x; i < total; i += kSortBlock) {
        const int64_t v = i / octs;
        const int c = (int)(i - v * octs) * kOct;
        store_n(p + v * a.table_stride + c, min(a.hidden - c, kOct), none);
    }
}

// Each sorted chunk's entries to their place in the whole list: what is below them
// in the other chunks (equal tokens of earlier chunks come first), first among the
// chunks' samples, in LDS, then in the stretch between two of them.  Eight chunks are
// searched at once, so that their loads wait together.
__global__ __launch_bounds__(kBlock) void merge_chunks_kernel(EmbeddingGradArgs a, int chunks)
{
    constexpr int Together = 8;
    extern __shared__ uint32_t samples[];   // chunks x kSamples
    for (int i = threadIdx.x; i < chunks * kSamples; i += kBlock)
        samples[i] = a.samples[i];
    __syncthreads();
    const int i = blockIdx.x * kBlock + threadIdx.x;
    if (i >= a.rows)
        return;
    const uint32_t x = a.chunk_key[i];
    const int own = i / a.chunk, stretch = a.chunk / kSamples;   // powers of two
    int place = i - own * a.chunk;
    for (int c0 = 0; c0 < chunks; c0 += Together) {
        int below[Together] = {}, size[Together];
        const uint32_t *keys[Together], *sample[Together];
        bool earlier[Together];
        auto is_below = [&](int t, uint32_t k) { return earlier[t] ? k <= x : k < x; };
#pragma unroll
        for (int t = 0; t < Together; ++t) {
            const int c = min(c0 + t, chunks - 1);
            keys[t] = a.chunk_key + c * a.chunk;
            sample[t] = samples + c * kSamples;
            size[t] = c0 + t < chunks && c != own ? min(a.rows - c * a.chunk, a.chunk) : 0;
            earlier[t] = c < own;
        }
        // samples below: by halves of them, and the last one
#pragma unroll
        for (int step = kSamples / 2; step >= 0; step = step > 0 ? step / 2 : -1) {
            uint32_t k[Together];
#pragma unroll
            for (int t = 0; t < Together; ++t)
                k[t] = sample[t][below[t] + max(step, 1) - 1];
#pragma unroll
            for (int t = 0; t < Together; ++t)
                below[t] += is_below(t, k[t]) ? max(step, 1) : 0;
        }
#pragma unroll
        for (int t = 0; t < Together; ++t)
            below[t] = size[t] ? below[t] * stretch : 0;
        for (int step = stretch / 2; step > 0; step /= 2) {
            uint32_t k[Together];
#pragma unroll
            for (int t = 0; t < Together; ++t)   // are the chunk's first below + step keys all below?
                k[t] = keys[t][min(below[t] + step, max(size[t], 1)) - 1];
#pragma unroll
            for (int t = 0; t < Together; ++t)
                if (below[t] + step <= size[t] && is_below(t, k[t]))
                    below[t] += step;
        }
#pragma unroll
        for (int t = 0; t < Together; ++t)
            place += below[t];
    }
    a.key[place] = x;
    a.row[place] = a.chunk_row[i];
}

// -- sums over sorted tokens -----------------------------------------------------------------

// The columns that a lane works on: eight from `from` on, of which n from element
// `shift` on are its own (at a row's end the last eight, behind it none of them; of a row
// of fewer than eight every lane works on all, the first lane has them).  Lanes that
// work on the same columns have the same sums, so where they store the same parts they
// store the same values.  whole: every lane of the wave has eight of its own.
struct Columns {
    int from, shift, n, hidden;
    bool whole;
    __device__ __forceinline__ Columns(int hidden_, int slab) : hidden(hidden_)
    {
        const int c = (slab * kWave + (int)threadIdx.x % kWave) * kOct;
        from = max(min(c, hidden - kOct), 0);
        shift = c - from;
        n = min(hidden - c, kOct);
        whole = (slab + 1) * kWave * kOct <= hidden;
    }
    template <typename T>
    __device__ __forceinline__ void load(const T *row, RawOct<T> &x) const
    {
        if (hidden < kOct)
            x.load(row, hidden);
        else
            x.load(row + from);
    }
};

// A token's finished sum to its row of the gradient, added to `was`, what is there,
// where accumulated.
template <typename O, bool ACC>
__device__ __forceinline__ void put(const EmbeddingGradArgs &a, O *row, const Columns &c, const float (&sum)[kOct],
                                    const RawOct<O> &was)
{
    float x[kOct];
#pragma unroll
    for (int k = 0; k < kOct; ++k)
        x[k] = ACC ? was.at(k) + a.scale * sum[k] : a.scale * sum[k];
    if (c.whole) {
        store8(row + c.from, x);
        return;
    }
#pragma unroll
    for (int k = 0; k < kOct; ++k)
        if (k >= c.shift && k < c.shift + c.n)
            row[c.from + k] = narrow<O>(x[k]);
}

__device__ __forceinline__ float *part_of(const EmbeddingGradArgs &a, int segment, int tail, int c)
{
    return a.parts + ((int64_t)segment * 2 + tail) * a.columns + c;
}

// A wave's segment and slab of 512 columns: neighbouring waves take a segment's slabs
// one after another, so that rows are read in long pieces.
__device__ __forceinline__ void unit_of(const EmbeddingGradArgs &a, int &segment, int &slab)
{
    const uint32_t u = __builtin_amdgcn_readfirstlane(blockIdx.x * (kBlock / kWave) + threadIdx.x / kWave);
    const uint32_t slabs = (uint32_t)(a.hidden + kOct * kWave - 1) / (kOct * kWave);
    segment = (int)(u / slabs), slab = (int)(u % slabs);
}

// Rows, and parts of a run, whose loads are on their way at once.
constexpr int kBatch = 8, kJoinBatch = 16;

// One wave per segment of the sorted list and 512 columns.  Lane e has the segment's
// entry e; what decides where sums end is in scalar registers.
template <typename T, typename O, bool ACC>
__global__ __launch_bounds__(kBlock) void segment_sum_kernel(EmbeddingGradArgs a)
{
    const int lane = threadIdx.x % kWave;
    int s, slab;
    unit_of(a, s, slab);
    if (s >= a.segments)
        return;
    const Columns c(a.hidden, slab);
    const int lo = s * a.segment, entries = min(a.segment, a.rows - lo);
    // the entries' tokens and rows, the tokens beside them (-1: none)
    const int e = lo + min(lane, entries - 1);
    const uint32_t key = a.key[e], row = a.row[e];
    const uint32_t before = lo > 0 ? a.key[lo - 1] : ~0u;
    const uint32_t after = lo + min(lane, entries - 1) + 1 < a.rows ? a.key[lo + min(lane, entries - 1) + 1] : ~0u;
    // entries that name a row, the last of each run among them, and whether the first
    // run began and the last goes on in other segments
    const uint64_t named = __ballot(lane < entries && key < (uint32_t)a.vocab);
    const int m = __popcll(named);
    if (m == 0)
        return;
    const uint64_t differ = __ballot(key != after);
    const uint64_t last = 1ull << (m - 1);
    const uint64_t ends = (differ & named) | last;
    const bool begun = __builtin_amdgcn_readfirstlane(before == key), goes_on = !(differ & last);
    bool first = true;
    float sum[kOct] = {};
    for (int e0 = 0; e0 < m; e0 += kBatch) {
        RawOct<T> x[kBatch];
        RawOct<O> was[kBatch];
        auto d_row = [&](int j) {
            return static_cast<O *>(a.d_table) + (int64_t)(uint32_t)__builtin_amdgcn_readlane(key, j) * a.table_stride;
        };
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int j = min(e0 + i, m - 1);
            c.load(static_cast<const T *>(a.d_out) + (int64_t)(uint32_t)__builtin_amdgcn_readlane(row, j) * a.stride, x[i]);
            if (ACC && (ends >> j & 1))
                c.load(d_row(j), was[i]);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int j = e0 + i;
            if (j < m) {
#pragma unroll
                for (int k = 0; k < kOct; ++k)
                    sum[k] += x[i].at(k);
                if (ends >> j & 1) {
                    const bool head = first && begun, tail = j == m - 1 && goes_on;
                    if (head || tail)
                        store8(part_of(a, s, !head, c.from), sum);
                    else
                        put<O, ACC>(a, d_row(j), c, sum, was[i]);
                    first = false;
#pragma unroll
                    for (int k = 0; k < kOct; ++k)
                        sum[k] = 0.0f;
                }
            }
        }
    }
}

// The runs that begin in a segment and go on in the next: a workgroup per segment and
// 512 columns, whose waves take a quarter each of the run's parts.
template <typename O, bool ACC>
__global__ __launch_bounds__(kBlock) void join_runs_kernel(EmbeddingGradArgs a)
{
    constexpr int Waves = kBlock / kWave;
    __shared__ f32x4 sh[Waves - 1][kWave][2];
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint32_t slabs = (uint32_t)(a.hidden + kOct * kWave - 1) / (kOct * kWave);
    const int s = (int)(blockIdx.x / slabs);
    const Columns c(a.hidden, (int)(blockIdx.x % slabs));
    const int lo = s * a.segment, next = lo + a.segment;
    const uint32_t run = a.key[next - 1], begins = a.key[next], before = lo > 0 ? a.key[lo - 1] : ~0u;
    if (run >= (uint32_t)a.vocab || begins != run || before == run)
        return;
    O *row = static_cast<O *>(a.d_table) + (int64_t)run * a.table_stride;
    RawOct<O> was;
    if (ACC && wave == 0)
        c.load(row, was);
    // the last segment that begins with the run: in steps that double, then halve
    int last = s + 1, step = 1;
    auto has = [&](int q) { return q < a.segments && a.key[q * a.segment] == run; };
    for (; has(last + step); step *= 2)
        last += step;
    for (step /= 2; step > 0; step /= 2)
        if (has(last + step))
            last += step;
    const int share = (last - s + 1 + Waves - 1) / Waves;   // parts s .. last, the first its segment's tail
    const int from = s + wave * share, to = min(from + share, last + 1);
    float sum[kOct] = {};
    for (int q = from; q < to; q += kJoinBatch) {
        float x[kJoinBatch][kOct];
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) {
            const int p = min(q + i, to - 1);
            load8(part_of(a, p, p == s, c.from), x[i]);
        }
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i)
            if (q + i < to)
#pragma unroll
                for (int k = 0; k < kOct; ++k)
                    sum[k] += x[i][k];
    }
    if (wave > 0)
        sh[wave - 1][lane][0] = f32x4{sum[0], sum[1], sum[2], sum[3]}, sh[wave - 1][lane][1] = f32x4{sum[4], sum[5], sum[6], sum[7]};
    __syncthreads();
    if (wave > 0)
        return;
#pragma unroll
    for (int w = 0; w < Waves - 1; ++w)
#pragma unroll
        for (int k = 0; k < kOct; ++k)
            sum[k] += sh[w][lane][k / 4][k % 4];
    put<O, ACC>(a, row, c, sum, was);
}

template <typename T, typename O>
void embedding_rows(const EmbeddingArgs &a, hipStream_t st)
{
    const uint32_t octs = (uint32_t)((a.hidden + kOct - 1) / kOct);
    const int64_t most = (int64_t(1) << 31) / octs;   // rows of a launch
    for (int64_t r = 0; r < a.rows; r += most) {
        const uint32_t total = (uint32_t)(std::min(most, a.rows - r) * octs);
        hipLaunchKernelGGL((embedding_kernel<T, O>), dim3((total + kBlock - 1) / kBlock), dim3(kBlock), 0, st, a,
                           r, octs, total);
    }
}

template <typename T, typename O>
void embedding_grad_of(const EmbeddingGradArgs &a, hipStream_t st)
{
    const int chunks = (a.rows + a.chunk - 1) / a.chunk;
    // octs of all rows, as the rows lie one after another or apart
    const int64_t octs = (int64_t)a.vocab * ((a.hidden + kOct - 1) / kOct);
    const int clear = a.accumulate ? 0 : (int)((octs + kClearOcts - 1) / kClearOcts);
    if (chunks + clear > 0)
        hipLaunchKernelGGL((sort_and_clear_kernel<O>), dim3(chunks + clear), dim3(kSortBlock), 0, st, a, chunks);
    if (a.rows == 0)
        return;
    const dim3 entries((a.rows + kBlock - 1) / kBlock);
    const size_t samples = chunks * kSamples * sizeof(uint32_t);
    if (chunks > 1)
        hipLaunchKernelGGL(merge_chunks_kernel, entries, dim3(kBlock), samples, st, a, chunks);
    const int64_t units = (int64_t)a.segments * ((a.hidden + kOct * kWave - 1) / (kOct * kWave));
    const dim3 grid((unsigned)((units + kBlock / kWave - 1) / (kBlock / kWave)));
    auto sums = [&](auto acc) {
        constexpr bool ACC = decltype(acc)::value;
        hipLaunchKernelGGL((segment_sum_kernel<T, O, ACC>), grid, dim3(kBlock), 0, st, a);
        if (a.segments > 1)   // the last segment's run goes on nowhere
            hipLaunchKernelGGL((join_runs_kernel<O, ACC>), dim3((unsigned)(units - units / a.segments)), dim3(kBlock), 0,
                               st, a);
    };
    if (a.accumulate)
        sums(std::true_type());
    else
        sums(std::false_type());
}

}  // namespace

// Eight rows wait for memory together, so a short segment is summed sooner, but a
// token of many rows leaves more parts to join.  Added to what is there, us, with
// segments of
//     rows x hidden        8    16    32    64
//     1024 x 1280         19    23    31    48
//     1000 x 5000         19    22    31    46
//    20000 x   64         45    43    48    64
//     8192 x 1280         38    39    45    64
//     4096 x 4096         38    38    42    55
//   100000 x   64        115    91    83    92
//    16384 x 4096         80    71    67    70
// Up to 32 rows are one segment, without a join.
int32_t embedding_segment(int64_t rows, int64_t hidden)
{
    static_assert(kOct * kWave == 512, "a slab");
    const int64_t work = rows * embedding_slabs(hidden);
    return rows <= 32 || work > kSegmentWork[1] ? 32 : work > kSegmentWork[0] ? 16 : 8;
}

int launch_embedding(const EmbeddingArgs &a, void *stream)
{
    by_types(a.dtype, a.out_dtype, [&](auto t, auto o) {
        embedding_rows<decltype(t), decltype(o)>(a, reinterpret_cast<hipStream_t>(stream));
    });
    return hipGetLastError();
}

int launch_embedding_grad(const EmbeddingGradArgs &a, void *stream)
{
    by_types(a.dtype, a.table_dtype, [&](auto t, auto o) {
        embedding_grad_of<decltype(t), decltype(o)>(a, reinterpret_cast<hipStream_t>(stream));
    });
    return hipGetLastError();
}

}  // namespace zero
