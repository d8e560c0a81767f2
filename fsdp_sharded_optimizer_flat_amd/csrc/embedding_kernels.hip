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
#include <algorithm>

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
constexpr int kPerThread = kSortChunk / kSortBlock;
static_assert(ZERO_MAX_VOCAB < 1 << (3 * kDigit), "a token and the mark of no token fit three digits");

struct SortShared {
    uint32_t key[kSortChunk];
    uint16_t at[kSortChunk];
    uint32_t count[kDigits * kSortWaves];   // [digit][wave]
    uint32_t wave_sum[kSortWaves];
};

// Sorts n <= kSortChunk tokens by value, stable, by digits from the lowest: a
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
}

// Elements of the gradient that a workgroup clears.
constexpr int kClearOcts = 8 * kSortBlock;

// The first `chunks` workgroups sort a chunk each, the others clear a span of the
// gradient each meanwhile (one after another in memory; with a share of the whole to
// each of as many as fit the device at once, the last of them started when the sorting
// was over: 175 us for 128256 x 4096 bf16, and 160 so).
template <typename T>
__global__ __launch_bounds__(kSortBlock) void sort_and_clear_kernel(EmbeddingGradArgs a, int chunks)
{
    __shared__ SortShared sh;
    if ((int)blockIdx.x < chunks) {
        const int first = blockIdx.x * kSortChunk;
        sort_chunk(a, first, min(a.rows - first, kSortChunk), sh);
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

// Number of keys in k[0..n) below x (or, with EQUAL, not above it).
template <bool EQUAL>
__device__ __forceinline__ int keys_below(const uint32_t *k, int n, uint32_t x)
{
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (EQUAL ? k[mid] <= x : k[mid] < x)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

// Each sorted chunk's entries to their place in the whole list: what is below them
// in the other chunks (equal tokens of earlier chunks come first).
__global__ __launch_bounds__(kBlock) void merge_chunks_kernel(EmbeddingGradArgs a, int chunks)
{
    const int i = blockIdx.x * kBlock + threadIdx.x;
    if (i >= a.rows)
        return;
    const uint32_t x = a.chunk_key[i];
    const int own = i / kSortChunk;
    int place = i - own * kSortChunk;
    for (int c = 0; c < chunks; ++c) {
        const int first = c * kSortChunk, n = min(a.rows - first, kSortChunk);
        if (c < own)
            place += keys_below<true>(a.chunk_key + first, n, x);
        else if (c > own)
            place += keys_below<false>(a.chunk_key + first, n, x);
    }
    a.key[place] = x;
    a.row[place] = a.chunk_row[i];
}

// -- sums over sorted tokens -----------------------------------------------------------------

// A token's finished sum to its row of the gradient, columns from c on: eight, or n of
// them from element `shift` on.
template <typename O>
__device__ __forceinline__ void put(const EmbeddingGradArgs &a, uint32_t token, int c, int shift, int n,
                                    const float (&sum)[kOct])
{
    O *p = static_cast<O *>(a.d_table) + (int64_t)token * a.table_stride + c;
    if (n >= kOct) {
        float x[kOct];
        if (a.accumulate)
            load8(p, x);
#pragma unroll
        for (int k = 0; k < kOct; ++k)
            x[k] = a.accumulate ? x[k] + a.scale * sum[k] : a.scale * sum[k];
        store8(p, x);
        return;
    }
#pragma unroll
    for (int k = 0; k < kOct; ++k)
        if (k >= shift && k < shift + n)
            p[k] = narrow<O>(a.accumulate ? widen<O>(p[k]) + a.scale * sum[k] : a.scale * sum[k]);
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

// Rows whose loads are on their way at once.
constexpr int kBatch = 8;

// One wave per segment of the sorted list and 512 columns.  Lane e has the segment's
// entry e.  A lane at the end of the columns takes the last eight, of which it stores
// those that are its own (rows of fewer than eight: element by element).
template <typename T, typename O>
__global__ __launch_bounds__(kBlock) void segment_sum_kernel(EmbeddingGradArgs a)
{
    const int lane = threadIdx.x % kWave;
    int s, slab;
    unit_of(a, s, slab);
    const int c = (slab * kWave + lane) * kOct, n = min(a.hidden - c, kOct);
    if (s >= a.segments)
        return;
    const int lo = s * a.segment, entries = min(a.segment, a.rows - lo);
    // the entries' tokens and rows, the tokens beside the segment (-1: none)
    const int e = lo + min(lane, entries - 1);
    const uint32_t key = a.key[e], row = a.row[e];
    const uint32_t before = lo > 0 ? a.key[lo - 1] : ~0u, after = lo + entries < a.rows ? a.key[lo + entries] : ~0u;
    const bool narrow_rows = a.hidden < kOct;
    const int from = narrow_rows ? 0 : min(c, a.hidden - kOct), shift = c - from;
    const T *d_out = static_cast<const T *>(a.d_out) + from;
    float sum[kOct] = {};
    uint32_t run = __builtin_amdgcn_readlane(key, 0);
    bool cut = before == run;
    for (int e0 = 0; e0 < entries; e0 += kBatch) {
        RawOct<T> x[kBatch];
        auto row_at = [&](int i) {
            return d_out + (int64_t)(uint32_t)__builtin_amdgcn_readlane(row, min(e0 + i, entries - 1)) * a.stride;
        };
        if (narrow_rows) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                x[i].load(row_at(i), n);
        } else {
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                x[i].load(row_at(i));
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int j = e0 + i;
            if (j >= entries || run >= (uint32_t)a.vocab)
                break;
#pragma unroll
            for (int k = 0; k < kOct; ++k)
                sum[k] += x[i].at(k);
            const uint32_t next = j + 1 < entries ? (uint32_t)__builtin_amdgcn_readlane(key, j + 1) : after;
            if (next == run && j + 1 < entries)
                continue;
            // the run ends here, or in another segment
            if (n > 0) {
                if (cut || next == run)
                    store8(part_of(a, s, !cut, from), sum);
                else
                    put<O>(a, run, from, shift, n, sum);
            }
            cut = false;
            run = next;
#pragma unroll
            for (int k = 0; k < kOct; ++k)
                sum[k] = 0.0f;
        }
    }
}

// The runs that begin in a segment and go on in the next: one wave per segment and
// 512 columns.
template <typename O>
__global__ __launch_bounds__(kBlock) void join_runs_kernel(EmbeddingGradArgs a)
{
    const int lane = threadIdx.x % kWave;
    int s, slab;
    unit_of(a, s, slab);
    const int c = (slab * kWave + lane) * kOct, n = min(a.hidden - c, kOct);
    if (s >= a.segments - 1 || n <= 0)
        return;
    const int lo = s * a.segment, next = lo + a.segment;
    const uint32_t run = a.key[next - 1], begins = a.key[next], before = lo > 0 ? a.key[lo - 1] : ~0u;
    if (run >= (uint32_t)a.vocab || begins != run || before == run)
        return;
    // the last segment that begins with the run: in steps that double, then halve
    int last = s + 1, step = 1;
    auto has = [&](int q) { return q < a.segments && a.key[q * a.segment] == run; };
    for (; has(last + step); step *= 2)
        last += step;
    for (step /= 2; step > 0; step /= 2)
        if (has(last + step))
            last += step;
    float sum[kOct], x[kBatch][kOct];
    load8(part_of(a, s, 1, c), sum);
    int q = s + 1;
    for (; q + kBatch <= last + 1; q += kBatch) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            load8(part_of(a, q + i, 0, c), x[i]);
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
#pragma unroll
            for (int k = 0; k < kOct; ++k)
                sum[k] += x[i][k];
    }
    for (; q <= last; ++q) {
        load8(part_of(a, q, 0, c), x[0]);
#pragma unroll
        for (int k = 0; k < kOct; ++k)
            sum[k] += x[0][k];
    }
    put<O>(a, run, c, 0, n, sum);
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
    const int chunks = (a.rows + kSortChunk - 1) / kSortChunk;
    // octs of all rows, as the rows lie one after another or apart
    const int64_t octs = (int64_t)a.vocab * ((a.hidden + kOct - 1) / kOct);
    const int clear = a.accumulate ? 0 : (int)((octs + kClearOcts - 1) / kClearOcts);
    if (chunks + clear > 0)
        hipLaunchKernelGGL((sort_and_clear_kernel<O>), dim3(chunks + clear), dim3(kSortBlock), 0, st, a, chunks);
    if (a.rows == 0)
        return;
    if (chunks > 1)
        hipLaunchKernelGGL(merge_chunks_kernel, dim3((a.rows + kBlock - 1) / kBlock), dim3(kBlock), 0, st, a,
                           chunks);
    const int64_t units = (int64_t)a.segments * ((a.hidden + kOct * kWave - 1) / (kOct * kWave));
    const dim3 grid((unsigned)((units + kBlock / kWave - 1) / (kBlock / kWave)));
    hipLaunchKernelGGL((segment_sum_kernel<T, O>), grid, dim3(kBlock), 0, st, a);
    if (a.segments > 1)
        hipLaunchKernelGGL((join_runs_kernel<O>), grid, dim3(kBlock), 0, st, a);
}

}  // namespace

int32_t embedding_segment(int64_t rows, int64_t hidden)
{
    const int64_t slabs = (hidden + kOct * kWave - 1) / (kOct * kWave);
    return rows > 32 && rows * slabs <= 32768 ? 8 : 32;
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
