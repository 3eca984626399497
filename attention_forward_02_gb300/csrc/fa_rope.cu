// fa_rope.cu -- host side of fa_rope declared in include/fa.h: argument checks
// and the launch.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "fa.h"
#include "fa_cache_host.h"
#include "fa_host.h"
#include "fa_rope_kernel.cuh"

namespace {

using namespace fa_host;

// A tensor of rows: its address, and (stride, extent) of batch, rows and heads.
struct View {
    uintptr_t at;
    long long batch, row, head;
    int B, N, H, d;

    size_t bytes() const
    {
        return static_cast<size_t>((B - 1) * batch + (N - 1) * row + (H - 1) * head + d) * 2;
    }
    // No element twice: each stride of a dimension spans the smaller ones.
    bool distinct() const
    {
        long long stride[3] = {batch, row, head}, span = d;
        int extent[3] = {B, N, H};
        for (int i = 0; i < 3; ++i)
            for (int j = i + 1; j < 3; ++j)
                if (stride[j] < stride[i]) {
                    const long long s = stride[i];
                    stride[i] = stride[j];
                    stride[j] = s;
                    const int e = extent[i];
                    extent[i] = extent[j];
                    extent[j] = e;
                }
        for (int i = 0; i < 3; ++i) {
            if (extent[i] == 1)
                continue;
            if (stride[i] < span)
                return false;
            span += (extent[i] - 1) * stride[i];
        }
        return true;
    }
};

// Where an element of one tensor lies from one of another: a sum of steps, `stride` times a number
// from lo to hi each.
struct Step {
    long long stride;
    int lo, hi;
};
constexpr int kSteps = 6;    // three dimensions of each
constexpr int kLooks = 4096;  // of the search below; a layout that needs more counts as overlapping

// Whether `at` and steps i .. n - 1, the largest strides first, come to between -d and d; rest_lo[i]
// and rest_hi[i] are the least and the most that steps from i on add.
bool reaches(const Step (&step)[kSteps], const long long (&rest_lo)[kSteps + 1], const long long (&rest_hi)[kSteps + 1], int i,
             int n, long long at, int d, int &looks)
{
    if (at + rest_hi[i] <= -d || at + rest_lo[i] >= d)
        return false;
    if (i == n || ++looks > kLooks)
        return true;
    for (long long x = step[i].lo; x <= step[i].hi; ++x) {
        // on to the first number that is not too low
        const long long short_of = -d + 1 - (at + x * step[i].stride + rest_hi[i + 1]);
        if (short_of > 0)
            x += (short_of + step[i].stride - 1) / step[i].stride;
        const long long next = at + x * step[i].stride;
        if (x > step[i].hi || next + rest_lo[i + 1] >= d)
            return false;
        if (reaches(step, rest_lo, rest_hi, i + 1, n, next, d, looks))
            return true;
    }
    return false;
}

// No element in common.  Different memory, as a rule; else the views' elements may lie between one
// another's: heads side by side in a row, a head's query, key and value side by side, heads of every batch.
// Along dimensions with one stride only the distance counts, so that the search tries two or three
// numbers for each.
bool apart(const View &a, const View &b)
{
    if (!overlaps(a.at, a.bytes(), b.at, b.bytes()))
        return true;
    const long long of_a[3] = {a.batch, a.row, a.head}, of_b[3] = {b.batch, b.row, b.head};
    const int ext_a[3] = {a.B, a.N, a.H}, ext_b[3] = {b.B, b.N, b.H};
    Step step[kSteps];
    int n = 0;
    const auto add = [&](long long stride, int lo, int hi) {
        if (stride == 0 || lo == hi)
            return;
        int i = n++;
        for (; i > 0 && step[i - 1].stride < stride; --i)
            step[i] = step[i - 1];
        step[i] = {stride, lo, hi};
    };
    for (int i = 0; i < 3; ++i) {
        if (of_a[i] == of_b[i]) {
            add(of_a[i], 1 - ext_b[i], ext_a[i] - 1);
        } else {
            add(of_a[i], 0, ext_a[i] - 1);
            add(of_b[i], 1 - ext_b[i], 0);
        }
    }
    long long rest_lo[kSteps + 1], rest_hi[kSteps + 1];
    rest_lo[n] = rest_hi[n] = 0;
    for (int i = n - 1; i >= 0; --i) {
        rest_lo[i] = rest_lo[i + 1] + step[i].lo * step[i].stride;
        rest_hi[i] = rest_hi[i + 1] + step[i].hi * step[i].stride;
    }
    int looks = 0;
    return !reaches(step, rest_lo, rest_hi, 0, n, static_cast<long long>(a.at - b.at) / 2, a.d, looks);
}

// Units of rows an SM below which a block shares its rows' sines (few heads share too little),
// and up to which, with a thread a unit, a row's heads are shared out: so that every SM has
// something, and, which leaves sixteen heads a thread, so that the last threads to start are few.
// Without the latter a second wave of few threads takes as long as the first: 12,000 rows of 40
// heads of 128 43.9 us on the GPU and 40.5 with it, 2 x 10,334 rows of 96 heads of 64 88.7 and
// 80.0, 30,000 97.2 and 94.0 (half as many units: 41.2, 79.6, 96.9).
constexpr int kFewUnits = 256, kFewHeads = 16, kUnits = 512, kManyUnits = 4096;

constexpr int kMaxHeads = 65535;

// Checks rows and fills their views; strides of dimensions of one become 0.
fa_status_t check_rows(fa_rope_rows_t &r, int B, int N, int d, View *x, View *y)
{
    long long *all[6] = {&r.x_batch, &r.y_batch, &r.x_row, &r.y_row, &r.x_head, &r.y_head};
    const int extent[3] = {B, N, r.heads};
    for (int i = 0; i < 6; ++i)
        if (extent[i / 2] == 1)
            *all[i] = 0;
    for (int i = 0; i < 6; ++i)
        if (!fine(*all[i], extent[i / 2]))
            return FA_ERR_INVALID_ARG;
    if (!r.x || !r.y)
        return FA_ERR_INVALID_ARG;
    long long bits = 0;
    for (const long long *s : all)
        bits |= *s;
    if ((u(r.x) | u(r.y)) & 15u || bits & 7)
        return FA_ERR_MISALIGNED;
    *x = {u(r.x), r.x_batch, r.x_row, r.x_head, B, N, r.heads, d};
    *y = {u(r.y), r.y_batch, r.y_row, r.y_head, B, N, r.heads, d};
    const bool in_place = r.x == r.y && r.x_batch == r.y_batch && r.x_row == r.y_row && r.x_head == r.y_head;
    if (!y->distinct() || !(in_place || apart(*x, *y)))
        return FA_ERR_INVALID_ARG;
    return FA_OK;
}

}  // namespace

extern "C" {

fa_status_t fa_rope(const fa_rope_t *rope, const fa_rope_rows_t *q, const fa_rope_rows_t *k, const int *positions,
                    long long position_stride, int B, int N, int d, int backward, fa_dtype_t dtype, void *stream)
{
    if (!rope || !q || B < 0 || N < 0 || q->heads < 0 || (k && k->heads < 0) || (backward != 0 && backward != 1) ||
        !std::isfinite(rope->factor) || (rope->interleaved != 0 && rope->interleaved != 1) || rope->pairs < 1)
        return FA_ERR_INVALID_ARG;
    if ((d != 32 && d != 64 && d != 96 && d != 128) || (dtype != FA_FP16 && dtype != FA_BF16) || rope->pairs % 4 != 0 ||
        rope->pairs > d / 2 || q->heads > kMaxHeads || (k && k->heads > kMaxHeads))
        return FA_ERR_UNSUPPORTED;
    const bool some_q = q->heads > 0, some_k = k && k->heads > 0;
    if (B == 0 || N == 0 || (!some_q && !some_k))
        return FA_OK;  // empty problem
    if (!rope->turns || (positions && !fine(position_stride, B)))
        return FA_ERR_INVALID_ARG;
    if (u(rope->turns) & 7u || u(positions) & 3u)
        return FA_ERR_MISALIGNED;
    if (B == 1)
        position_stride = 0;
    fa_rope_rows_t rows[2] = {*q, k ? *k : fa_rope_rows_t()};
    View x[2], y[2];
    const uintptr_t at[2] = {u(rope->turns), u(positions)};
    const size_t bytes[2] = {static_cast<size_t>(rope->pairs) * 8,
                             positions ? static_cast<size_t>((B - 1) * position_stride + N) * 4 : 0};
    for (int i = 0; i < 2; ++i) {
        if (!(i ? some_k : some_q))
            continue;
        const fa_status_t s = check_rows(rows[i], B, N, d, &x[i], &y[i]);
        if (s != FA_OK)
            return s;
        for (int j = 0; j < 2; ++j)
            if (bytes[j] && overlaps(y[i].at, y[i].bytes(), at[j], bytes[j]))
                return FA_ERR_INVALID_ARG;
    }
    if (some_q && some_k && !(apart(y[0], y[1]) && apart(y[0], x[1]) && apart(y[1], x[0])))
        return FA_ERR_INVALID_ARG;
    int sms = 0;
    fa_host::EncodeTiledFn encode = nullptr;
    const fa_status_t s = fa_host::encoder(&encode, &sms);
    if (s != FA_OK)
        return s;
    const long long total = static_cast<long long>(B) * N;
    const int heads = (some_q ? rows[0].heads : 0) + (some_k ? rows[1].heads : 0);
    const int units = d / 8, places = fa::rope::kThreads / units;  // of a block: rows times slots
    if (total * units > 0x7fffffffLL / 2)
        return FA_ERR_UNSUPPORTED;
    fa::rope::Rows r[2];
    for (int i = 0; i < 2; ++i)
        r[i] = {rows[i].x,      rows[i].y,     rows[i].x_batch, rows[i].x_head, rows[i].x_row,
                rows[i].y_batch, rows[i].y_head, rows[i].y_row,   (i ? some_k : some_q) ? rows[i].heads : 0};
    const fa::rope::Turn turn = {rope->turns, rope->pairs, rope->factor, backward == 1};
    fa::rope::Shape shape = {positions, position_stride, static_cast<unsigned>(N), static_cast<unsigned>(total), units, 1};
    dim3 grid(1);
    const bool few = total * units < static_cast<long long>(sms) * kFewUnits && heads >= kFewHeads;
    if (few) {
        while (shape.slots < 8 && 4 * shape.slots < heads && 2 * shape.slots <= places)
            shape.slots *= 2;
        const int per_block = places / shape.slots;
        grid.x = static_cast<unsigned>((total + per_block - 1) / per_block);
        while (static_cast<long long>(grid.y) * shape.slots < heads && static_cast<long long>(grid.x) * grid.y < sms)
            grid.y *= 2;
    } else {
        // more threads than the GPU holds at once, but sixteen heads for each pair's sine, if there are so many
        const auto below = [&](int per_sm) { return total * units * shape.slots < static_cast<long long>(sms) * per_sm; };
        while ((shape.slots < heads && below(kUnits)) || (heads >= 16 * shape.slots && below(kManyUnits)))
            shape.slots *= 2;
        grid.x = static_cast<unsigned>((total * units * shape.slots + fa::rope::kThreads - 1) / fa::rope::kThreads);
    }
    const auto of_type = [&](auto t) {
        using T = decltype(t);
        using namespace fa::rope;
        const auto kernel = few ? (rope->interleaved ? fa_rope_rows_kernel<T, true> : fa_rope_rows_kernel<T, false>)
                                : (rope->interleaved ? fa_rope_kernel<T, true> : fa_rope_kernel<T, false>);
        return launch_dependent(kernel, grid, kThreads, 0, static_cast<cudaStream_t>(stream), r[0], r[1], turn, shape)
                   ? launched()
                   : FA_ERR_CUDA;
    };
    return dtype == FA_FP16 ? of_type(__half()) : of_type(__nv_bfloat16());
}

}  // extern "C"
