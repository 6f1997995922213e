// Which rows the experts of a grouped product have and how the workers share its
// tiles (gemm_grouped.cu); host code too, so that it can be checked without a GPU.
#pragma once

#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

namespace fp8k {
namespace grouped {

// An expert's rows: its two bounds cut to 0 .. R, the end no lower than the begin.
struct Bounds {
    int begin, end;
    bool back;  // the second bound is below the first
};
__host__ __device__ __forceinline__ Bounds bounds_within(int lo, int hi, int R) {
    const int begin = lo < 0 ? 0 : lo < R ? lo : R;
    const int end = hi < 0 ? 0 : hi < R ? hi : R;
    return {begin, end < begin ? begin : end, end < begin};
}

// Where bounds go back, each counts as the largest up to it, so that no row has two
// experts and the experts' tiles stay as many as R rows can have.
__host__ __device__ inline void put_in_order(int* begin, int* end, int E) {
    int most = 0;
    for (int e = 0; e < E; ++e) {
        begin[e] = most = begin[e] < most ? most : begin[e];
        end[e] = most = end[e] < most ? most : end[e];
    }
}

// A worker's pieces of the list in order: whole tiles, then its share of the
// tiles that are cut.
//
// The last round is cut where that is sooner done.  With `rest` tiles left it
// takes nk stages of
//   u(w) = max(stage, w shared) us with w workers busy
// (what one SM can load, what the card can; for tiles bound by the tensor cores
// `shared` is 0).  Cut into equal shares for m workers it takes rest nk / m stages
// of u(m), and the join of the parts, `fixed` + `part` for each of a tile's.
// sqrt(nk stage / part) parts a tile balance the shares with the join.
struct Costs {
    float stage, shared, fixed, part;
    __host__ __device__ __forceinline__ float round(int busy) const {
        return fmaxf(stage, busy * shared);
    }
};
struct Walk {
    int workers, nk;         // workers of the cut tiles
    int whole;               // tiles of the list that are taken whole
    int64_t units;           // stages of the others
    int next;
    int64_t u, u_end;
    int tile, kb0, kb1;
    __host__ __device__ __forceinline__ Walk(int all, int n, int me, int stages, const Costs& c)
        : workers(0), nk(stages), whole(all), units(0), next(me), step(n) {
        const int rest = all % n;
        if (rest) {
            const int m = static_cast<int>(fminf(static_cast<float>(n), rest * sqrtf(nk * c.stage / c.part)));
            if (m > rest && static_cast<float>(nk) * rest / m * c.round(m) + c.fixed + c.part * (static_cast<float>(m) / rest + 1.0f) <
                                nk * c.round(rest)) {
                whole = all - rest;
                units = static_cast<int64_t>(rest) * nk;
                workers = units < m ? static_cast<int>(units) : m;  // (a stage for each at least)
            }
        }
        u = me < workers ? units * me / workers : 0;
        u_end = me < workers ? units * (me + 1) / workers : 0;
    }
    __host__ __device__ __forceinline__ bool advance() {
        if (next < whole) {
            tile = next;
            kb0 = 0, kb1 = nk;
            next += step;
            return true;
        }
        if (u >= u_end) return false;
        const int64_t j = u / nk;
        tile = whole + static_cast<int>(j);
        kb0 = static_cast<int>(u - j * nk);
        kb1 = kb0 + (u_end - u) < nk ? static_cast<int>(kb0 + (u_end - u)) : nk;
        u += kb1 - kb0;
        return true;
    }
    // the worker that has unit x of the cut tiles
    __host__ __device__ __forceinline__ int worker_of(int64_t x) const {
        return static_cast<int>(((x + 1) * workers - 1) / units);
    }

   private:
    int step;
};

}  // namespace grouped
}  // namespace fp8k
