// rows_kernels.hpp -- kernels of the calls around products whose B is picked
// row by row: the router and its gradient, the slots sorted by group, the
// weighted sum of a token's slots and its gradient, and the products in their
// simplest form (any strides; the fast forms are in grouped_kernels.hpp).
#pragma once

#include "lanes.hpp"

namespace rowk {

// ---------------------------------------------------------------------------
// The router.  L lanes hold one row: element e = l + L v in register v of lane
// l, so a load instruction covers 64 / L rows' contiguous pieces.  The k
// choices are k rounds of an arg-max over the row: the lanes' own maxima, a
// reduction over the L lanes, then the lowest index among the lanes that hold
// the maximum; the owner's element is then taken out.
//
// What decides the order is a sum of scores (a bias, or the two best of a
// group), where 32 bits would swap neighbours that differ by less than their
// rounding: WIDE computes scores and keys in 64 bits.  Otherwise the scores
// rise with the logits, and those are compared as they are.  The chosen
// weights (one lane per choice), and a softmax row's sum, are computed in 64 bits
// either way and rounded once.
//
// The instructions issued bound it where there is a bias: 8191 x 256 with 8 groups
// takes 11.4 us (8.4 MB of logits: 2), of which the 64-bit exponentials and the 8
// rounds are a third each.  16384 x 64, k 6, without: 4.8 us renormalised and 5.5
// with the row's sum (5.1 in 32 bits), of which 2.2 are the launch.
// ---------------------------------------------------------------------------
struct RouteArgs {
    int T, E, k, sigmoid, groups, top_groups, group_best, renorm;
    float scale, inv_per;  // inv_per: 1 / (E / groups)
    const float *logits, *bias;
    int64_t ldl;
    int *ids;
    float *weights;
};

// exp(x - m) with m the row's maximum; equal values (infinities too) give 1.
// (No branches here or below: around each element they kept the elements' loads
// and exponentials from overlapping.)
__device__ __forceinline__ double exp_below(double x, double m) { return exp(x == m ? 0.0 : x - m); }

constexpr int kRouteThreads = 256;

// A key that stands for nothing, and taking a key out: of a double the upper
// half alone is replaced, which leaves at most -1.79e308.
template <class Key> constexpr Key kNothing = -INFINITY;
template <> constexpr double kNothing<double> = -1.79e308;
__device__ __forceinline__ bool something(float key) { return key > -INFINITY; }
__device__ __forceinline__ bool something(double key) { return key > -1.78e308; }
__device__ __forceinline__ void take_out(float &key, bool it) { key = it ? -INFINITY : key; }
__device__ __forceinline__ void take_out(double &key, bool it) {
    key = __hiloint2double(it ? (int)0xffefffff : __double2hiint(key), __double2loint(key));
}

// k rounds of an arg-max over the L V keys of a row, element l + L v in register
// v of lane l; lane j keeps the j-th choice, or -1.
template <int L, int V, class Key> __device__ __forceinline__ int choose(Key (&key)[V], int k, int l) {
    int mine = -1;
    for (int j = 0; j < k; ++j) {
        Key best = key[0];
#pragma unroll
        for (int v = 1; v < V; ++v) best = fmax(best, key[v]);
        const Key most = reduce<L>(best, Max());
        int at[V];  // (apart, so that no compare waits for the select before it)
#pragma unroll
        for (int v = 0; v < V; ++v) at[v] = key[v] == most ? l + L * v : INT_MAX;
#pragma unroll
        for (int n = V; n > 1; n = (n + 1) / 2)
#pragma unroll
            for (int v = 0; v < n / 2; ++v) at[v] = Min()(at[v], at[n - 1 - v]);
        const int first = reduce<L>(something(most) ? at[0] : INT_MAX, Min());
#pragma unroll
        for (int v = 0; v < V; ++v) take_out(key[v], l + L * v == first);
        if (l == j) mine = first == INT_MAX ? -1 : first;
    }
    return mine;
}

template <int L, int V, bool WIDE>
__global__ void __launch_bounds__(kRouteThreads) route(RouteArgs a) {
    typedef typename std::conditional<WIDE, double, float>::type Key;
    constexpr int ROWS = kRouteThreads / L;
    constexpr Key NONE = kNothing<Key>;
    constexpr int GROUPS = L * V < 64 ? L * V : 64;  // at most
    __shared__ Key keys[ROWS][L * V + L * V / 32 + 1];
    __shared__ Key worth[ROWS][GROUPS];
    __shared__ int kept[ROWS][GROUPS];
    const int l = threadIdx.x % L, r = threadIdx.x / L;
    const int t = (int)blockIdx.x * ROWS + r;
    const bool in = t < a.T;
    const float *row = a.logits + (int64_t)(in ? t : 0) * a.ldl;

    float x[V], bias[V];
    float top = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = row[l + L * v < a.E ? l + L * v : 0];
    if (WIDE && a.bias != nullptr) {
#pragma unroll
        for (int v = 0; v < V; ++v) bias[v] = a.bias[l + L * v < a.E ? l + L * v : 0];
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) bias[v] = 0.0f;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        x[v] = in && l + L * v < a.E ? x[v] : -INFINITY;
        nan |= x[v] != x[v];
        top = fmaxf(top, x[v]);  // a NaN is passed over
    }
    top = reduce<L>(top, Max());
    const int bad = reduce<L>(nan ? 0 : 1, Min());  // 0: some logit of the row is NaN

    Key key[V];
    double total = 0.0;
    if constexpr (WIDE) {
        if (a.sigmoid) {
#pragma unroll
            for (int v = 0; v < V; ++v) key[v] = 1.0 / (1.0 + exp(-(double)x[v]));
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                key[v] = exp_below((double)x[v], (double)top);
                key[v] = x[v] > -INFINITY ? key[v] : 0.0;
                total += key[v];
            }
            total = reduce<L>(total, Add());
#pragma unroll
            for (int v = 0; v < V; ++v) key[v] /= total;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const double s = key[v] + (double)bias[v];
            key[v] = x[v] > -INFINITY && s > NONE ? s : NONE;  // (neither NaN nor -inf)
        }
    } else {
        if (!a.sigmoid && !a.renorm) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const double p = exp_below((double)x[v], (double)top);
                total += x[v] > -INFINITY ? p : 0.0;
            }
            total = reduce<L>(total, Add());
        }
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = x[v] > -INFINITY ? x[v] : NONE;
    }

    int mine;  // lane j keeps choice j
    if (a.groups > 1) {
        // Each group's worth from the keys in LDS: a lane per group (the rows of 32
        // keys a bank apart), or the row's lanes together where groups are long.  A
        // group is kept when fewer than top_groups are worth more (or as much, with
        // a lower index).
        const int per = a.E / a.groups;
        auto place = [](int e) { return e + (e >> 5); };
#pragma unroll
        for (int v = 0; v < V; ++v) keys[r][place(l + L * v)] = key[v];
        __syncthreads();
        // the two highest of two pairs, b0 >= b1 and q0 >= q1
        auto join = [](Key &b0, Key &b1, Key q0, Key q1) {
            b1 = fmax(fmin(b0, q0), fmax(b1, q1));
            b0 = fmax(b0, q0);
        };
        // (no sum where the second is missing)
        auto value = [&](Key b0, Key b1) { return a.group_best == 2 && something(b1) ? b0 + b1 : b0; };
        if (per > 4 * L) {
            for (int g = 0; g < a.groups; ++g) {
                Key b0 = NONE, b1 = NONE;
                for (int i = l; i < per; i += L) join(b0, b1, keys[r][place(g * per + i)], NONE);
                join(b0, b1, dpp<0x128>(b0), dpp<0x128>(b1));
                join(b0, b1, dpp<0x124>(b0), dpp<0x124>(b1));
                join(b0, b1, dpp<0x122>(b0), dpp<0x122>(b1));
                join(b0, b1, dpp<0x121>(b0), dpp<0x121>(b1));
                if constexpr (L == 64) {
                    Key c0 = at_lane(b0, 0), c1 = at_lane(b1, 0);
                    for (int i = 16; i < 64; i += 16) join(c0, c1, at_lane(b0, i), at_lane(b1, i));
                    b0 = c0;
                    b1 = c1;
                }
                if (l == 0) worth[r][g] = value(b0, b1);
            }
        } else {
            for (int g = l; g < a.groups; g += L) {
                Key b0 = NONE, b1 = NONE;
#pragma unroll 8
                for (int i = 0; i < per; ++i) {
                    const Key q = keys[r][place(g * per + i)];
                    b1 = fmax(b1, fmin(b0, q));
                    b0 = fmax(b0, q);
                }
                worth[r][g] = value(b0, b1);
            }
        }
        __syncthreads();
        // the kept groups in their order, and with them their elements
        for (int g = l; g < a.groups; g += L) {
            const Key w = worth[r][g];
            int above = 0;
            for (int h = 0; h < a.groups; ++h) {
                const Key o = worth[r][h];
                above += (o > w || (o == w && h < g)) ? 1 : 0;
            }
            kept[r][g] = above < a.top_groups ? 1 : 0;
        }
        __syncthreads();
        int place_of[GROUPS / L > 0 ? GROUPS / L : 1];
#pragma unroll
        for (int i = 0; i < GROUPS / L; ++i) {
            int n = 0;
            for (int h = 0; h < l + L * i && h < a.groups; ++h) n += kept[r][h];
            place_of[i] = l + L * i < a.groups && kept[r][l + L * i] ? n : -1;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < GROUPS / L; ++i)
            if (place_of[i] >= 0) kept[r][place_of[i]] = l + L * i;
        __syncthreads();
        const int count = a.top_groups * per;
        auto element = [&](int i) {
            // exact: i < 1024, and (i + 1/2) / per is at least 1 / (2 per) from a whole number
            const int q = (int)(((float)i + 0.5f) * a.inv_per);
            return kept[r][q] * per + (i - q * per);
        };
        auto some = [&](auto registers) __attribute__((always_inline)) {
            constexpr int VV = decltype(registers)::value;
            Key left[VV];
#pragma unroll
            for (int v = 0; v < VV; ++v) {
                const int i = l + L * v;
                const Key q = keys[r][place(element(i < count ? i : 0))];
                left[v] = i < count ? q : NONE;
            }
            return choose<L>(left, a.k, l);
        };
        if (count <= L * (V / 2)) mine = some(std::integral_constant<int, V / 2 ? V / 2 : 1>());
        else mine = some(std::integral_constant<int, V>());
        if (mine >= 0) mine = element(mine);
    } else {
        mine = choose<L>(key, a.k, l);
    }

    const bool found = mine >= 0;
    const float xm = found ? row[mine] : -INFINITY;
    double s;
    if (a.sigmoid) {
        s = 1.0 / (1.0 + exp(-(double)xm));
    } else {
        // renormalised over the chosen alone: their own maximum, so that far
        // choices do not vanish
        const float m = a.renorm ? reduce<L>(xm, Max()) : top;
        s = exp_below((double)xm, (double)m);
        if (!a.renorm) s /= total;
    }
    if (!found) s = 0.0;
    if (a.renorm) {
        const double sum = reduce<L>(s, Add());
        s = sum > 0.0 ? s / sum : 0.0;
    }
    if (in && l < a.k) {
        a.ids[(int64_t)t * a.k + l] = mine;
        a.weights[(int64_t)t * a.k + l] = !found ? 0.0f : bad == 0 ? NAN : (float)(s * (double)a.scale);
    }
}

// ---------------------------------------------------------------------------
// The router's gradient, from the logits, the ids and the weights' gradient c
// (scaled): with p the weights before `scale`,
//   renorm:  dl_i = p_i (c_i - sum c p) for the chosen (times 1 - s_i for the
//            sigmoid), 0 elsewhere; the rest of the row need not be read;
//   else softmax: dl_e = s_e (c_e - sum c s), sigmoid: dl_e = c_e s_e (1 - s_e).
// A confident router has a weight next to 1, and c_i - sum c p cancels there (to 0
// in 32 bits from a gap of 17 between the logits).  So b, the c of the highest
// logit (0 where that is not chosen), is taken off first: of the sum's terms
// p_i (c_i - b) the large one is then 0 exactly, and
//   c_e - sum c p = (c_e - b) - sum p_i (c_i - b),
// the last sum over the chosen with renorm, else over the row, where what was not
// chosen gives -b times the sum of the scores beside the highest.  All in 64 bits,
// rounded once, one lane per choice, spread over the row through LDS.
// 16384 x 64, k 6, takes 5.0 us, of which 2.2 are the launch and 1.7 the 8.4 MB (4.1
// with the row in 32 bits); 4096 x 1024 12.5 (9.2).  Chosen alone (renorm): 3.9.
// ---------------------------------------------------------------------------
struct RouteGradArgs {
    int T, E, k, sigmoid, renorm;
    float scale;
    const float *logits;
    int64_t ldl;
    const int *ids;
    const float *dweights;
    float *dlogits;
    int64_t lddl;
};

template <int L, int V>
__global__ void __launch_bounds__(kRouteThreads) route_grad(RouteGradArgs a) {
    constexpr int ROWS = kRouteThreads / L;
    __shared__ double spread[ROWS][L * V + 1];
    const int l = threadIdx.x % L, r = threadIdx.x / L;
    const int t = (int)blockIdx.x * ROWS + r;
    const bool in = t < a.T;
    const float *row = a.logits + (int64_t)(in ? t : 0) * a.ldl;
    const bool whole = !a.sigmoid && !a.renorm;  // every element has a gradient

    int id = -1;
    double c = 0.0;
    if (in && l < a.k) {
        id = a.ids[(int64_t)t * a.k + l];
        if ((unsigned)id >= (unsigned)a.E) id = -1;
        if (id >= 0) c = (double)a.dweights[(int64_t)t * a.k + l] * (double)a.scale;
    }
    const float xi = id >= 0 ? row[id] : -INFINITY;
    const bool has = xi > -INFINITY || xi != xi;

    // whole: the row's exponentials, their sum `rest` where the logit is not the
    // highest, and how many are the highest
    double e[V], rest = 0.0, ties = 0.0;
    float top = -INFINITY;
    if (whole) {
        float x[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            x[v] = in && l + L * v < a.E ? row[l + L * v] : -INFINITY;
            top = fmaxf(top, x[v]);
        }
        top = reduce<L>(top, Max());
#pragma unroll
        for (int v = 0; v < V; ++v) {
            e[v] = exp_below((double)x[v], (double)top);
            e[v] = x[v] == -INFINITY ? 0.0 : e[v];
            rest += x[v] == top ? 0.0 : e[v];
            ties += x[v] == top && x[v] > -INFINITY ? 1.0 : 0.0;
        }
        rest = reduce<L>(rest, Add());
        ties = reduce<L>(ties, Add());
    } else {
        top = reduce<L>(xi, Max());
    }
    const int first = reduce<L>(has && xi == top ? l : INT_MAX, Min());  // a choice of the highest logit
    const double b = reduce<L>(l == first ? c : 0.0, Add());

    double d;          // the chosen expert's gradient; whole: what its score multiplies
    double off = 0.0;  // whole: what the other experts' scores multiply
    if (whole) {
        const double sum = rest + ties, inv = sum == 0.0 ? 0.0 : 1.0 / sum;
        const double s = has ? exp_below((double)xi, (double)top) : 0.0;
        double q = reduce<L>(l == first ? 0.0 : s * c, Add());
        if (first != INT_MAX) q -= b * (rest + (ties - 1.0));
        q *= inv;
        d = (c - b) - q;
        off = -b - q;
#pragma unroll
        for (int v = 0; v < V; ++v) e[v] *= inv;
    } else {
        double s = 0.0, other = 1.0;
        if (a.sigmoid) {
            if (has) s = 1.0 / (1.0 + exp(-(double)xi));
            other = 1.0 / (1.0 + exp((double)xi));  // 1 - s without cancellation
        } else if (has) {
            s = exp_below((double)xi, (double)top);
        }
        if (a.renorm) {
            const double S = reduce<L>(s, Add());
            const double p = S != 0.0 ? s / S : 0.0;
            d = p * ((c - b) - reduce<L>(id >= 0 ? p * (c - b) : 0.0, Add())) * other;
        } else {
            d = c * s * other;
        }
    }

#pragma unroll
    for (int v = 0; v < V; ++v) spread[r][l + L * v] = off;
    __syncthreads();
    if (id >= 0) spread[r][id] = d;
    __syncthreads();
    if (!in) return;
    float *out = a.dlogits + (int64_t)t * a.lddl;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int at = l + L * v;
        if (at >= a.E) continue;
        const double w = spread[r][at];
        out[at] = (float)(whole ? e[v] * w : w);
    }
}

// ---------------------------------------------------------------------------
// Slots sorted by group: a counting sort that keeps the slots' order.  4096 slots
// at a time, each of a workgroup's waves taking a run of consecutive ones, 64 to a
// register.  The place of a slot is: where its group begins, plus the group's
// slots in earlier runs, plus those earlier in its own run; these are counted with
// one ballot per bit of the id (the lanes whose ids agree in every bit), so there is
// no atomic and the order is the slots' own.  One workgroup does it all up to 4096
// slots; beyond, a first launch counts each workgroup's slots and in a second
// every workgroup adds up what lies before its own.  Latency bounds it: 4022 slots
// take 7 us (13 with the ids read again from memory), 8192 in two launches 12.
// ---------------------------------------------------------------------------
constexpr int kGroupSlots = 4096;

struct GroupArgs {
    int R, G, run;  // run: slots per workgroup, whole turns of kGroupSlots
    const int *ids;
    int *offsets, *rows, *counts;  // counts: [workgroups][G]
};

// lanes with the same id
__device__ __forceinline__ unsigned long long same_id(int id, int bits) {
    unsigned long long m = ~0ull;
    for (int b = 0; b < bits; ++b) {
        const unsigned long long set = __ballot((id >> b) & 1);
        m &= (id >> b) & 1 ? set : ~set;
    }
    return m;
}

template <int GMAX, int WAVES, bool COUNT_ONLY>
__global__ void __launch_bounds__(64 * WAVES) group_rows(GroupArgs a) {
    constexpr int NT = 64 * WAVES, PER = kGroupSlots / NT, GROUPS = GMAX / NT;
    static_assert(PER * NT == kGroupSlots && GROUPS * NT == GMAX, "whole registers, whole groups per thread");
    __shared__ int count[WAVES][GMAX];
    __shared__ int wave_sum[WAVES];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int nwg = gridDim.x, wg = blockIdx.x;
    const int64_t begin = (int64_t)wg * a.run, end = begin + a.run < a.R ? begin + a.run : a.R;
    const int bits = 32 - __clz(a.G);  // ids up to G itself, which stands for none
    const unsigned long long below = (1ull << lane) - 1;

    int id[PER], before[PER];  // a slot's id, and its group's slots earlier in the wave's run
    auto read = [&](int64_t from) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int64_t s = from + (w * PER + i) * 64 + lane;
            id[i] = s < end ? a.ids[s] : a.G;
            if ((unsigned)id[i] >= (unsigned)a.G) id[i] = a.G;
        }
    };
    auto tally = [&]() {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const unsigned long long same = same_id(id[i], bits);
            int n = 0;
            if (id[i] < a.G) n = count[w][id[i]];  // every lane reads before the first one writes
            __builtin_amdgcn_wave_barrier();
            if (id[i] < a.G && (same & below) == 0) count[w][id[i]] = n + __popcll(same);
            __builtin_amdgcn_wave_barrier();
            before[i] = n + __popcll(same & below);
        }
    };
    auto clear = [&]() {
        for (int i = lane; i < a.G; i += 64) count[w][i] = 0;
    };

    if constexpr (COUNT_ONLY) {
        clear();
        for (int64_t from = begin; from < end; from += kGroupSlots) {
            read(from);
            tally();
        }
        __syncthreads();
        for (int g = tid; g < a.G; g += NT) {
            int n = 0;
#pragma unroll
            for (int i = 0; i < WAVES; ++i) n += count[i][g];
            a.counts[(int64_t)wg * a.G + g] = n;
        }
        return;
    }

    read(begin);
    clear();
    tally();
    __syncthreads();
    // thread i takes GROUPS consecutive groups: their totals, what earlier
    // workgroups hold of them, and the sum of all lower ones
    int at[GROUPS], total[GROUPS], sum = 0;
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
        const int g = tid * GROUPS + i;
        total[i] = at[i] = 0;
        if (g < a.G) {
            if (nwg == 1) {
#pragma unroll
                for (int j = 0; j < WAVES; ++j) total[i] += count[j][g];
            } else {
                for (int b = 0; b < nwg; ++b) {
                    const int n = a.counts[(int64_t)b * a.G + g];
                    total[i] += n;
                    at[i] += b < wg ? n : 0;
                }
            }
        }
        sum += total[i];
    }
    int upto = sum;  // inclusive over the wave's lanes
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(upto, d);
        if (lane >= d) upto += o;
    }
    if (lane == 63) wave_sum[w] = upto;
    __syncthreads();
    int base = upto - sum;
    for (int i = 0; i < w; ++i) base += wave_sum[i];
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
        const int g = tid * GROUPS + i;
        if (g >= a.G) break;
        if (wg == 0) {
            a.offsets[g] = base;
            if (g == a.G - 1) a.offsets[a.G] = base + total[i];
        }
        at[i] += base;
        base += total[i];
    }
    for (int64_t from = begin;;) {
        // each wave's first place in every group
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) {
            const int g = tid * GROUPS + i;
            if (g >= a.G) break;
#pragma unroll
            for (int j = 0; j < WAVES; ++j) {
                const int n = count[j][g];
                count[j][g] = at[i];
                at[i] += n;
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (id[i] < a.G) a.rows[count[w][id[i]] + before[i]] = (int)(from + (w * PER + i) * 64 + lane);
        from += kGroupSlots;
        if (from >= end) break;
        read(from);
        clear();  // (the wave's own counts, which it alone has just read)
        tally();
        __syncthreads();
    }
}

// Up to 64 slots (a token or two): one wave, a slot per lane, every place
// counted from the other lanes' ids.
__global__ void __launch_bounds__(64) group_few(GroupArgs a) {
    const int lane = threadIdx.x;
    int id = a.G;
    if (lane < a.R) {
        id = a.ids[lane];
        if ((unsigned)id >= (unsigned)a.G) id = a.G;
    }
    int place = 0;
    for (int j = 0; j < a.R; ++j) {
        const int o = at_lane(id, j);
        place += (o < id || (o == id && j < lane)) ? 1 : 0;
    }
    if (id < a.G) a.rows[place] = lane;
    for (int g = lane; g <= a.G; g += 64) {
        int n = 0;
        for (int j = 0; j < a.R; ++j) n += at_lane(id, j) < g ? 1 : 0;
        a.offsets[g] = n;
    }
}

// ---------------------------------------------------------------------------
// A row times its own adapter's U (K x rank), for few rows: a workgroup of 256 per
// row and piece of K, four columns per lane, the lanes of a column group taking k
// in turn; H holds the pieces' sums, [piece][row][rank].  And back: a wave per row
// and 256 columns adds alpha s h V_g to C.  Memory bounds both (29 rows with an
// adapter each, rank 64: 15 MB of U in 5.1 us, 30 MB of V in 8.0, launches in it);
// loads go through descriptors that end where the data does, because a branch
// around each kept them from overlapping (V took 28 us), and V's first rows are on
// their way while h is summed (29 rows 22.0 us in all, 22.7 with h first).
// ---------------------------------------------------------------------------
struct ShrinkArgs {
    int M, K, G, rank, parts;
    const float *A, *U;
    int64_t lda, ldu, stride_u;
    const int *ids, *ranks;
    float *H;
};

__device__ __forceinline__ void shrink_row(const ShrinkArgs &a, int block) {
    __shared__ __attribute__((aligned(16))) float part[256 * 4];
    const int m = block % a.M, piece = block / a.M;
    if (piece >= a.parts) return;
    const int id = a.ids[m];
    if ((unsigned)id >= (unsigned)a.G) return;
    int rank = a.rank;
    if (a.ranks != nullptr) {
        rank = a.ranks[id];
        rank = rank < 0 ? 0 : (rank > a.rank ? a.rank : rank);
    }
    int quads = 1;  // column groups, rounded up to a power of two: at most 64
    while (4 * quads < rank) quads *= 2;
    const int tid = threadIdx.x, q = tid % quads, kl = tid / quads, step = 256 / quads;
    const int k0 = (int)((int64_t)a.K * piece / a.parts), k1 = (int)((int64_t)a.K * (piece + 1) / a.parts);
    // what lies past the piece's last k reads 0.0 (and columns past the rank, which
    // go on into the next row, are not written)
    const rsrc_t ra = whole_rsrc(a.A + (int64_t)m * a.lda + k0, (int64_t)(k1 - k0) * 4);
    const rsrc_t ru = whole_rsrc(a.U + (int64_t)id * a.stride_u + (int64_t)k0 * a.ldu,
                                 ((int64_t)(k1 - k0 - 1) * a.ldu + rank) * 4);
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    if (4 * q < rank) {
        for (int k = kl; k < k1 - k0; k += 8 * step) {  // eight in flight
            f32x4 u[8];
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t at = (uint32_t)(k + i * step);
                u[i] = sgk::raw_load_v4f32(ru, (at * (uint32_t)a.ldu + 4u * (uint32_t)q) * 4u, 0, 0);
                x[i] = sgk::raw_load_f32(ra, at * 4u, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) acc = fma4(x[i], u[i], acc);
        }
    }
    *reinterpret_cast<float4 *>(&part[4 * tid]) = make_float4(acc.x, acc.y, acc.z, acc.w);
    for (int half = step / 2; half > 0; half /= 2) {  // pairs, always in the same order
        __syncthreads();
        if (kl < half) {
            float4 &x = *reinterpret_cast<float4 *>(&part[4 * tid]);
            const float4 y = *reinterpret_cast<const float4 *>(&part[4 * (tid + half * quads)]);
            x.x += y.x;
            x.y += y.y;
            x.z += y.z;
            x.w += y.w;
        }
    }
    __syncthreads();
    if (tid < rank) a.H[((int64_t)piece * a.M + m) * a.rank + tid] = part[tid];
}

struct ExpandArgs {
    int M, N, G, rank, parts, chunks;  // chunks of 256 columns
    float alpha;
    const float *H, *V, *scales;
    int64_t ldv, stride_v, ldc;
    const int *ids, *ranks;
    float *C;
};

__global__ void __launch_bounds__(64) expand_rows(ExpandArgs a) {
    constexpr int DEEP = 16;  // rows of V in flight
    __shared__ float h[256];
    const int m = blockIdx.x / a.chunks, lane = threadIdx.x;
    const int c0 = (int)(blockIdx.x % a.chunks) * 256;  // first column
    const int id = a.ids[m];
    if ((unsigned)id >= (unsigned)a.G) return;
    int rank = a.rank;
    if (a.ranks != nullptr) {
        rank = a.ranks[id];
        rank = rank < 0 ? 0 : (rank > a.rank ? a.rank : rank);
    }
    if (rank == 0) return;
    const int64_t bytes = (int64_t)(a.N - c0) * 4;
    const uint32_t off = 16u * (uint32_t)lane;
    const rsrc_t rc = whole_rsrc(a.C + (int64_t)m * a.ldc + c0, bytes);
    const float *V = a.V + (int64_t)id * a.stride_v + c0;
    f32x4 v[DEEP];
    auto fetch = [&](int k) {  // rows past the rank read 0.0, as h does
#pragma unroll
        for (int i = 0; i < DEEP; ++i)
            v[i] = sgk::raw_load_v4f32(whole_rsrc(V + (int64_t)(k + i) * a.ldv, k + i < rank ? bytes : 0), off, 0, 0);
    };
    f32x4 acc = sgk::raw_load_v4f32(rc, off, 0, 0);
    fetch(0);  // on its way while h is summed
    const float s = a.scales != nullptr ? a.alpha * a.scales[id] : a.alpha;
    for (int k = lane; k < (rank + DEEP - 1) / DEEP * DEEP; k += 64) {
        float x = 0.0f;
        if (k < rank) {
#pragma unroll 16
            for (int i = 0; i < a.parts; ++i) x += a.H[((int64_t)i * a.M + m) * a.rank + k];
        }
        h[k] = k < rank ? s * x : 0.0f;
    }
    __syncthreads();
    for (int k = 0;;) {
#pragma unroll
        for (int i = 0; i < DEEP; ++i) acc = fma4(h[k + i], v[i], acc);
        k += DEEP;
        if (k >= rank) break;
        fetch(k);
    }
    sgk::raw_store_v4f32(acc, rc, off, 0, 0);
}

// ---------------------------------------------------------------------------
// The weighted sum of a token's k slots: one wave per 256 columns of a token,
// 16 bytes per lane and slot, four slots' loads in flight.  4096 tokens x 2 x 4096
// take 33 us, 6.1 TB/s: memory.
// ---------------------------------------------------------------------------
struct CombineArgs {
    int T, k, N, E;
    const int *ids;
    const float *weights, *Y;
    int64_t ldy, ldo;
    float beta;
    float *out;
    int chunks;  // of 256 columns
    int64_t units;
};

__global__ void __launch_bounds__(256) combine(CombineArgs a) {
    const int64_t unit = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    if (unit >= a.units) return;
    const int t = (int)(unit / a.chunks), c0 = (int)(unit - (int64_t)t * a.chunks) * 256;
    const int64_t s0 = (int64_t)t * a.k, bytes = (int64_t)(a.N - c0) * 4;
    const uint32_t off = 16u * (threadIdx.x & 63);
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j0 = 0; j0 < a.k; j0 += 4) {
        f32x4 y[4];
        float w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t s = s0 + (j0 + j < a.k ? j0 + j : 0);
            const bool there = j0 + j < a.k && (a.ids == nullptr || (unsigned)a.ids[s] < (unsigned)a.E);
            w[j] = !there ? 0.0f : a.weights == nullptr ? 1.0f : a.weights[s];
            // a slot that is not there reads 0.0 from an empty descriptor
            y[j] = sgk::raw_load_v4f32(whole_rsrc(a.Y + s * a.ldy + c0, there ? bytes : 0), off, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) acc = fma4(w[j], y[j], acc);
    }
    const rsrc_t ro = whole_rsrc(a.out + (int64_t)t * a.ldo + c0, bytes);
    if (a.beta != 0.0f) acc = fma4(a.beta, sgk::raw_load_v4f32(ro, off, 0, 0), acc);
    sgk::raw_store_v4f32(acc, ro, off, 0, 0);
}

// Its gradient: a workgroup per token, dout read once per eight slots (2011 x 2 x
// 2048: 19 us, 4.3 TB/s; a token's sums end in a barrier that the next slots wait for).
struct CombineGradArgs {
    int T, k, N, E;
    const int *ids;
    const float *weights, *dout, *Y;
    int64_t ldd, ldy, lddy;
    float *dY, *dweights;
};

__global__ void __launch_bounds__(256) combine_grad(CombineGradArgs a) {
    constexpr int J = 8;
    __shared__ float part[4][J];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int t = blockIdx.x;
    const bool dots = a.dweights != nullptr, rows = a.dY != nullptr;
    for (int j0 = 0; j0 < a.k; j0 += J) {
        const int nj = a.k - j0 < J ? a.k - j0 : J;
        const int64_t s0 = (int64_t)t * a.k + j0;
        float dot[J], wt[J];
        bool there[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            dot[j] = 0.0f;
            there[j] = j < nj && (a.ids == nullptr || (unsigned)a.ids[s0 + (j < nj ? j : 0)] < (unsigned)a.E);
            wt[j] = !there[j] ? 0.0f : a.weights == nullptr ? 1.0f : a.weights[s0 + j];
        }
        for (int c0 = 0; c0 < a.N; c0 += 1024) {
            const int64_t bytes = (int64_t)(a.N - c0) * 4;
            const uint32_t off = 16u * (uint32_t)tid;
            const f32x4 d = sgk::raw_load_v4f32(whole_rsrc(a.dout + (int64_t)t * a.ldd + c0, bytes), off, 0, 0);
            f32x4 y[J];
#pragma unroll
            for (int j = 0; j < J; ++j)  // (nothing is read through an empty descriptor)
                if (dots && j < nj)
                    y[j] = sgk::raw_load_v4f32(whole_rsrc(a.Y + (s0 + j) * a.ldy + c0, there[j] ? bytes : 0), off, 0, 0);
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (rows && j < nj) {
                    f32x4 g = {0.0f, 0.0f, 0.0f, 0.0f};
                    if (there[j]) {
                        g.x = wt[j] * d.x;
                        g.y = wt[j] * d.y;
                        g.z = wt[j] * d.z;
                        g.w = wt[j] * d.w;
                    }
                    sgk::raw_store_v4f32(g, whole_rsrc(a.dY + (s0 + j) * a.lddy + c0, bytes), off, 0, 0);
                }
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (dots && there[j])
                    dot[j] = fmaf(d.x, y[j].x, fmaf(d.y, y[j].y, fmaf(d.z, y[j].z, fmaf(d.w, y[j].w, dot[j]))));
        }
        if (a.dweights == nullptr) continue;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const float s = reduce<64>(dot[j], Add());
            if (lane == 0) part[w][j] = s;
        }
        __syncthreads();
        if (tid < nj) a.dweights[s0 + tid] = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Products over groups of rows: what every form of them is given.
// ---------------------------------------------------------------------------
struct GroupedArgs {
    int G, R;       // offsets NULL: one group of all R rows
    int N, K;       // tn: C_g is M x N
    int M;          // tn only
    float alpha, beta;
    const float *A, *B;
    float *C;
    int64_t lda, ldb, ldc, stride_b, stride_c;
    int a_div, b_div, c_scatter;
    const int *offsets, *rows;
    // adapters: a factor per group, and the part of K (NN, NT), of N or of M
    // (tn: C's columns or rows beyond it get no contribution) that a group has
    const float *scales;
    const int *ranks;
    int rank_k, rank_n, rank_m;
    int xcd_shift;  // log2 of the device's XCDs
};

__device__ __forceinline__ int clamp_to(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

__device__ __forceinline__ void group_range(const GroupedArgs &a, int g, int &p0, int &p1) {
    p0 = 0;
    p1 = a.R;
    if (a.offsets != nullptr) {
        p0 = clamp_to(a.offsets[g], 0, a.R);
        p1 = clamp_to(a.offsets[g + 1], 0, a.R);
    }
}

// The group and first row of a launch's t-th tile of `bm` rows, groups in
// order, each taking ceil(rows / bm) tiles.  A wave looks at 64 groups at a
// time (each lane one), so every wave of a workgroup finds it by itself.
// False: there are fewer tiles.
__device__ __forceinline__ bool find_tile(const GroupedArgs &a, int bm, int t, int &g, int &p0, int &p1) {
    const int lane = threadIdx.x & 63;
    const int groups = a.offsets != nullptr ? a.G : 1;
    for (int base = 0; base < groups; base += 64) {
        int lo = 0, hi = 0;
        if (base + lane < groups) group_range(a, base + lane, lo, hi);
        const int n = hi > lo ? (hi - lo + bm - 1) / bm : 0;
        int upto = n;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(upto, d);
            if (lane >= d) upto += o;
        }
        const unsigned long long past = __ballot(upto > t);
        if (past != 0) {
            const int at = __ffsll((long long)past) - 1;
            const int first = __builtin_amdgcn_readlane(upto - n, at);
            g = base + at;
            p0 = __builtin_amdgcn_readlane(lo, at) + (t - first) * bm;
            p1 = __builtin_amdgcn_readlane(hi, at);
            return true;
        }
        t -= __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}

// the rows of an operand that R slots reach (unsigned: R + div - 1 passes 31 bits)
__device__ __forceinline__ int64_t rows_behind(int R, int div) {
    return div > 1 ? ((unsigned)R + (unsigned)div - 1u) / (unsigned)div : (unsigned)R;
}

// place p's row of an operand: p itself, or rows[p] / div; -1: no such slot
__device__ __forceinline__ int64_t row_of(const GroupedArgs &a, int p, int div) {
    if (div == 0) return p;
    const int s = a.rows[p];
    if ((unsigned)s >= (unsigned)a.R) return -1;
    return div == 1 ? s : s / div;
}

// C's row of place p: none where the place's slot is asked for and is not one
__device__ __forceinline__ int64_t c_row_of(const GroupedArgs &a, int p) {
    if (a.a_div == 0 && a.c_scatter == 0) return p;
    const int64_t slot = row_of(a, p, 1);
    return slot < 0 || a.c_scatter != 0 ? slot : p;
}

__device__ __forceinline__ float group_alpha(const GroupedArgs &a, int g) {
    return a.scales != nullptr ? a.alpha * a.scales[g] : a.alpha;
}
__device__ __forceinline__ int group_rank(const GroupedArgs &a, int g, int whole) {
    return a.ranks != nullptr ? clamp_to(a.ranks[g], 0, whole) : whole;
}

// The simplest form, for operands that the fast ones do not take (offsets
// beyond 32 bits): 32 x 32 of C per workgroup, 64-bit addresses, every access
// checked.
template <bool TRANS_B>
__global__ void __launch_bounds__(256) grouped_simple(GroupedArgs a) {
    constexpr int T = 32;
    __shared__ float As[T][T + 1], Bs[T][T + 1];
    const int ncol = (a.N + T - 1) / T;
    const int n0 = (int)(blockIdx.x % ncol) * T;
    int g, p0, p1;
    if (!find_tile(a, T, (int)(blockIdx.x / ncol), g, p0, p1)) return;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const float *B = a.B + (int64_t)g * a.stride_b;
    const int K = a.rank_k ? group_rank(a, g, a.K) : a.K;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k0 = 0; k0 < K; k0 += T) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty + 8 * i;
            const int p = p0 + r;
            const int64_t ar = p < p1 ? row_of(a, p, a.a_div) : -1;
            As[r][tx] = ar >= 0 && k0 + tx < K ? a.A[ar * a.lda + k0 + tx] : 0.0f;
            const int bk = TRANS_B ? k0 + tx : k0 + r, bn = TRANS_B ? n0 + r : n0 + tx;
            const float b = bk < K && bn < a.N ? B[TRANS_B ? (int64_t)bn * a.ldb + bk : (int64_t)bk * a.ldb + bn] : 0.0f;
            if (TRANS_B) Bs[tx][r] = b;
            else Bs[r][tx] = b;
        }
        __syncthreads();
        for (int k = 0; k < T; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = fmaf(As[ty + 8 * i][k], Bs[k][tx], acc[i]);
        __syncthreads();
    }
    const float al = group_alpha(a, g);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int p = p0 + ty + 8 * i;
        if (p >= p1 || n0 + tx >= a.N) continue;
        const int64_t cr = c_row_of(a, p);
        if (cr < 0) continue;
        float *q = a.C + cr * a.ldc + n0 + tx;
        *q = a.beta != 0.0f ? fmaf(a.beta, *q, al * acc[i]) : al * acc[i];
    }
}

__global__ void __launch_bounds__(256) grouped_tn_simple(GroupedArgs a) {
    constexpr int T = 32;
    __shared__ float As[T][T + 1], Bs[T][T + 1];
    const int nm = (a.M + T - 1) / T, nn = (a.N + T - 1) / T;
    const int g = (int)(blockIdx.x / ((int64_t)nm * nn));
    const int rest = (int)(blockIdx.x - (int64_t)g * nm * nn);
    const int m0 = rest / nn * T, n0 = rest % nn * T;
    int p0, p1;
    group_range(a, g, p0, p1);
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int q0 = p0; q0 < p1; q0 += T) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty + 8 * i, p = q0 + r;
            const int64_t ar = p < p1 ? row_of(a, p, a.a_div) : -1;
            const int64_t br = p < p1 ? row_of(a, p, a.b_div) : -1;
            As[r][tx] = ar >= 0 && br >= 0 && m0 + tx < a.M ? a.A[ar * a.lda + m0 + tx] : 0.0f;
            Bs[r][tx] = ar >= 0 && br >= 0 && n0 + tx < a.N ? a.B[br * a.ldb + n0 + tx] : 0.0f;
        }
        __syncthreads();
        for (int k = 0; k < T; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = fmaf(As[k][ty + 8 * i], Bs[k][tx], acc[i]);
        __syncthreads();
    }
    const float al = group_alpha(a, g);
    const int mr = a.rank_m ? group_rank(a, g, a.M) : a.M, nr = a.rank_n ? group_rank(a, g, a.N) : a.N;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = m0 + ty + 8 * i, n = n0 + tx;
        if (m >= a.M || n >= a.N) continue;
        float *q = a.C + (int64_t)g * a.stride_c + (int64_t)m * a.ldc + n;
        const float v = m < mr && n < nr ? al * acc[i] : 0.0f;
        *q = a.beta != 0.0f ? fmaf(a.beta, *q, v) : v;
    }
}

}  // namespace rowk
