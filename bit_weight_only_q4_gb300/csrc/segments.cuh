// Sequences that are packed one behind the other: rows offsets[b] .. offsets[b + 1] - 1 belong to
// sequence b.  Lengths are read on the device; their work is cut into units that are numbered
// through, and a warp finds a unit by its number.
#pragma once

#include "q4_device.cuh"
#include "q4_internal.h"

namespace q4 {

struct Segments {
    const int32_t *offsets;      // [batch + 1]
    int batch, rows;             // rows: those there are
    int span, times;             // a sequence of n rows has ceil(n / span) * times units
    unsigned *err;
};

struct SegmentUnit {
    int sequence, start, len;    // the sequence, its first row and rows
    int unit;                    // unit of it, 0 ..
};

// Finds units by their number, at little cost when it rises from one to the next.  A warp takes the sequences 32 at a time, and asks
// for the next 32 offsets before it adds up those at hand.  Offsets that fall: a sequence that would begin before
// the end of one in front of it is left out, so that no row is written twice and the work stays
// bounded whatever the offsets are.
struct SegmentWalk {
    const Segments s;
    int chunk, base, total, floor;         // first sequence of the 32 at hand, units before them and among them; rows taken
    int start, len, before;                // this lane's sequence, units before it among the 32
    int next_lo, next_hi;

    __device__ explicit SegmentWalk(const Segments &segments)
        : s(segments), chunk(-32), base(0), total(0), floor(0), start(0), len(0), before(0)
    {
        ask(0);
    }

    __device__ void ask(int first)
    {
        const int b = first + (int)(threadIdx.x & 31);
        next_lo = first < s.batch && b < s.batch ? __ldg(s.offsets + b) : 0;
        next_hi = first < s.batch && b < s.batch ? __ldg(s.offsets + b + 1) : 0;
    }

    __device__ bool find(int number, SegmentUnit &u)
    {
        const int lane = threadIdx.x & 31;
        if (number < base) {                   // back to the front
            chunk = -32;
            base = total = floor = 0;
            ask(0);
        }
        while (number >= base + total) {
            if (chunk >= s.batch - 32)             // (no more: the walk stays where it is)
                return false;
            base += total;
            chunk += 32;
            int lo = next_lo, hi = next_hi;
            if (chunk < s.batch - 32)
                ask(chunk + 32);
            const bool here = chunk < s.batch - lane;
            const bool outside = lo < 0 || hi < 0 || lo > s.rows || hi > s.rows;
            lo = lo < 0 ? 0 : lo > s.rows ? s.rows : lo;
            hi = hi < 0 ? 0 : hi > s.rows ? s.rows : hi;
            int top = hi;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int v = __shfl_up_sync(0xffffffffu, top, o);
                top = lane >= o && v > top ? v : top;
            }
            int under = __shfl_up_sync(0xffffffffu, top, 1);
            under = lane > 0 && under > floor ? under : floor;
            const bool bad = here && (hi < lo || lo < under);
            if (here && (bad || outside) && s.err)
                atomicOr(s.err, kErrIndex);
            start = lo;
            len = bad || !here ? 0 : hi - lo;
            const int all = __shfl_sync(0xffffffffu, top, 31);
            floor = all > floor ? all : floor;
            const int units = (len / s.span + (len % s.span != 0)) * s.times;
            int sum = units;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int v = __shfl_up_sync(0xffffffffu, sum, o);
                sum += lane >= o ? v : 0;
            }
            before = sum - units;
            total = __shfl_sync(0xffffffffu, sum, 31);
        }
        const int at = number - base;
        const int src = 31 - __clz(__ballot_sync(0xffffffffu, before <= at));
        u.sequence = chunk + src;
        u.start = __shfl_sync(0xffffffffu, start, src);
        u.len = __shfl_sync(0xffffffffu, len, src);
        u.unit = at - __shfl_sync(0xffffffffu, before, src);
        return true;
    }
};

}  // namespace q4
