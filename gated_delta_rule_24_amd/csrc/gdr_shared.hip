// Attention of one query token per sequence over the paged 8-bit cache, where groups
// of sequences share their first pages (samples and beams of one prompt, a common
// system prompt).
//
//   o = sum_j p_j v_j / sum_j p_j, p_j = exp2(s_j - m), s_j = scale log2(e) q.k_j
//
// over the last `window` of a sequence's cached tokens (all: window 0).  A softmax over
// the shared pages and one over a sequence's own join as partial results do: each keeps
// its maximum m, its sum of exp2(s - m) and its unnormalised output.  So the
// shared pages are read once for the rows (a sequence's query heads on a key head) of
// the whole group, as further columns of the products that one sequence's heads
// already share in gdr_attn_decode.
#include "gdr_device.h"
#include "gdr_attn.h"
#include "gdr_attn_tile.h"
#include "gdr_generation.h"
#include "gdr_kv_tile.h"

namespace gdr {

namespace {

constexpr int kPage = 64;
constexpr int kWaves = 4;

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }

// first and one past the last cached token that a sequence's query sees
__device__ __forceinline__ void seen_range(const SharedParams& p, int n, int& lo, int& hi) {
    const long long room = (long long)p.max_pages * kPage;
    const int len = p.cache_len[n];
    hi = len < 0 ? 0 : (int)(len > room ? room : len);
    lo = (p.window > 0 && len > p.window) ? min(len - p.window, hi) : 0;
}

// A group's sequences first .. end - 1 and the pages they share; no content of the two
// arrays leads out of the tensors.
struct Group {
    int first, end, pages;
};
__device__ __forceinline__ Group group_at(const SharedParams& p, int g) {
    Group x;
    x.first = clampi(p.group_start[g], 0, p.N);
    x.end = clampi(p.group_start[g + 1], x.first, p.N);
    x.pages = clampi(p.shared_pages[g], 0, p.max_pages);
    return x;
}

// The group of tile `tile`, where a group of S sequences has ceil(S rows / width)
// tiles, and the tile's number in it; false behind the last.  All lanes together: 64
// groups are one load each.
__device__ __forceinline__ bool group_of_tile(const SharedParams& p, int rows, int width, int tile, int lane, int& g, int& t) {
    int before = 0;
    for (int g0 = 0; g0 < p.groups; g0 += 64) {
        int cnt = 0;
        if (g0 + lane < p.groups) {
            const Group x = group_at(p, g0 + lane);
            cnt = (int)(((long long)(x.end - x.first) * rows + width - 1) / width);
        }
        int run = cnt;
        for (int o = 1; o < 64; o <<= 1) {
            const int y = __shfl_up(run, o, 64);
            if (lane >= o) run += y;
        }
        const uint64_t m = __ballot(before + run > tile);
        if (m) {
            const int l = __builtin_ctzll(m);
            g = g0 + l;
            t = tile - before - (__builtin_amdgcn_readlane(run, l) - __builtin_amdgcn_readlane(cnt, l));
            return true;
        }
        before += __builtin_amdgcn_readlane(run, 63);
    }
    return false;
}

// The pages that sequence n shares with its group; 0 if it is in none.
__device__ __forceinline__ int shared_pages_of(const SharedParams& p, int n, int lane) {
    int s = 0, count = p.groups;                      // the last start <= n is among s .. s + count - 1, if it is anywhere
    while (count > 64) {
        const int step = (count + 63) / 64, i = s + lane * step;
        const uint64_t m = __ballot(lane * step < count && p.group_start[i] <= n);
        const int k = m ? 63 - __builtin_clzll(m) : 0;
        s += k * step;
        count = min(step, count - k * step);
    }
    const uint64_t m = __ballot(lane < count && p.group_start[s + lane] <= n);
    if (!m) return 0;
    const Group x = group_at(p, s + 63 - __builtin_clzll(m));
    return n >= x.first && n < x.end ? x.pages : 0;
}

__device__ __forceinline__ void store_out(const SharedParams& p, size_t idx, float x) {
    if (p.flags & GDR_OUT_BF16) reinterpret_cast<uint16_t*>(p.o)[idx] = f32_to_bf16(x);
    else reinterpret_cast<float*>(p.o)[idx] = x;
}

// e4m3 bytes that are NaN (0x7f, 0xff), as 0x80 in their places
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

}  // namespace

// One workgroup: the rows (columns of the products) of a tile of a group, or of one
// sequence's own pages, over a run of pages; its waves take pages in turn, each
// with its own running maximum and sum, and join at the end.  NC sets of 16 columns.
//
// The scores S^T[key][row] and the output O^T[channel][row] are laid out as in
// attn_decode_kernel: a lane has the keys 16 g .. 16 g + 15 of its column.  A weight is
// exp2(s - m); for the product with v it is taken times 2^(15 + log2 v_scale + m - wm), wm
// the running maximum of s + log2 v_scale, so that it has its f16 bits whatever the
// pages' scales: as the sum of two f16 values (22 bits) for fp32 results, as one
// (11 bits) for bf16 ones, whose own rounding is 8 times that.
template <int D, int NC, int PARTS>
__global__ __launch_bounds__(64 * kWaves) void attn_shared_kernel(SharedParams p) {
    constexpr int KS = D / 64;                        // 64-channel steps of a key row
    constexpr int VT = D / 16;                        // 16-channel tiles of the output
    __shared__ float s_o[kWaves][16][D + 4];
    __shared__ float s_ml[kWaves][16][2];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = lane & 15, g = lane >> 4;
    const int rep = p.Hq / p.Hkv;

    // which rows: row0 .. row0 + rows - 1 of a key head, row r being query head r % rep of
    // sequence `first` + r / rep; which pages: run `slot` of them, in sequence `first`'s table
    int first, row0, rows, kh, slot, pg0, pg1, table_row;
    const int shared_items = p.tiles * p.Hkv * p.shared_splits;
    if ((int)blockIdx.x < shared_items) {
        int unit, tile, gi;
        attn::work_item(blockIdx.x, p.Hkv * p.shared_splits, p.tiles, unit, tile);
        kh = unit % p.Hkv;
        slot = unit / p.Hkv;
        if (!group_of_tile(p, rep, 16 * NC, tile, lane, gi, tile)) return;
        const Group x = group_at(p, gi);
        if (x.pages == 0) return;                     // (the join reads no shared part then)
        first = x.first;
        table_row = first;
        row0 = 16 * NC * tile;
        rows = min(16 * NC, (x.end - x.first) * rep - row0);
        // the shared pages that some row of the group sees
        int lo = INT_MAX, hi = 0;
        for (int n = x.first + lane; n < x.end; n += 64) {
            int a, b;
            seen_range(p, n, a, b);
            if (a < b) { lo = min(lo, a); hi = max(hi, b); }
        }
        for (int o = 32; o > 0; o >>= 1) { lo = min(lo, __shfl_xor(lo, o, 64)); hi = max(hi, __shfl_xor(hi, o, 64)); }
        pg0 = lo / kPage;
        pg1 = min((int)(((long long)hi + kPage - 1) / kPage), x.pages);
        const int per = max(pg1 > pg0 ? (pg1 - pg0 + p.shared_splits - 1) / p.shared_splits : 0, kWaves);
        pg0 = pg1 > pg0 ? min(pg0 + slot * per, pg1) : pg1;
        pg1 = min(pg0 + per, pg1);
    } else {
        int w = blockIdx.x - shared_items;
        const int groups = (rep + 16 * NC - 1) / (16 * NC);
        const int qg = w % groups; w /= groups;
        kh = w % p.Hkv; w /= p.Hkv;
        first = w % p.N;
        slot = p.shared_splits + w / p.N;
        table_row = first;
        row0 = 16 * NC * qg;
        rows = min(16 * NC, rep - row0);
        int lo, hi;
        seen_range(p, first, lo, hi);
        pg0 = max(lo / kPage, shared_pages_of(p, first, lane));
        pg1 = (int)(((long long)hi + kPage - 1) / kPage);
        const int per = max(pg1 > pg0 ? (pg1 - pg0 + p.own_splits - 1) / p.own_splits : 0, kWaves);
        const int i = w / p.N;
        pg0 = pg1 > pg0 ? min(pg0 + i * per, pg1) : pg1;
        pg1 = min(pg0 + per, pg1);
    }
    const int sets = (rows + 15) / 16;

    // queries: column `col` of set c, channels 64 s + 16 g + 8 half ..
    bf8v qf[NC][KS][2];
    int lo[NC], hi[NC];                               // keys that the column sees
    int lo_most = 0, hi_least = INT_MAX, hi_most = 0, lo_least = INT_MAX;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int r = row0 + 16 * c + col;
        const bool live = 16 * c + col < rows;
        lo[c] = 0; hi[c] = 0;
        if (live) {
            seen_range(p, first + r / rep, lo[c], hi[c]);
            lo_most = max(lo_most, lo[c]);
            hi_least = min(hi_least, hi[c]);
            lo_least = min(lo_least, lo[c]);
            hi_most = max(hi_most, hi[c]);
        }
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                uint4 u = make_uint4(0, 0, 0, 0);
                if (live)
                    u = *reinterpret_cast<const uint4*>((const uint16_t*)p.q + ((size_t)(first + r / rep) * p.Hq + kh * rep + r % rep) * D +
                                                        64 * s + 16 * g + 8 * hf);
                qf[c][s][hf] = __builtin_bit_cast(bf8v, u);
            }
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) {
        lo_most = max(lo_most, __shfl_xor(lo_most, o, 64));
        hi_least = min(hi_least, __shfl_xor(hi_least, o, 64));
        lo_least = min(lo_least, __shfl_xor(lo_least, o, 64));
        hi_most = max(hi_most, __shfl_xor(hi_most, o, 64));
    }

    float4v o[NC][VT];
    float m[NC], l[NC], wm[NC];                       // maximum and sum of the scores; maximum of the weights
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        m[c] = -INFINITY; l[c] = 0.f; wm[c] = -INFINITY;
#pragma unroll
        for (int i = 0; i < VT; ++i) o[c][i] = float4v{0.f, 0.f, 0.f, 0.f};
    }
    const float to2 = p.scale * 1.4426950408889634f;
    const int krow = 16 * (col >> 2) + (col & 3);     // key of tile 0's row `col`

    for (int pg = pg0 + wave; pg < pg1; pg += kWaves) {
        int page = p.block_table[(size_t)table_row * p.max_pages + pg];
        const int at0 = pg * kPage;
        const bool absent = (unsigned)page >= (unsigned)p.n_pages;
        if (absent) page = 0;
        const size_t ph = (size_t)page * p.Hkv + kh;
        const uint8_t* kp = p.k_cache + ph * (kPage * D);
        const uint8_t* vp = p.v_cache + ph * (kPage * D);
        uint4 kk[4][KS], vv[VT];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int s = 0; s < KS; ++s)
                kk[t][s] = *reinterpret_cast<const uint4*>(kp + (krow + 4 * t) * D + 64 * s + 16 * g);
#pragma unroll
        for (int i = 0; i < VT; ++i)
            vv[i] = *reinterpret_cast<const uint4*>(vp + (size_t)(g * D + 16 * i + col) * 16);
        const float ks = p.k_scale[ph] * to2, vs = __builtin_amdgcn_logf(p.v_scale[ph]);   // base 2

        float4v sc[NC][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
#pragma unroll
            for (int c = 0; c < NC; ++c) sc[c][t] = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const bf8v k0 = e4m3x8_to_bf16(kk[t][s].x, kk[t][s].y), k1 = e4m3x8_to_bf16(kk[t][s].z, kk[t][s].w);
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    if (c == 0 || c < sets) {
                        sc[c][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k0, qf[c][s][0], sc[c][t], 0, 0, 0);
                        sc[c][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k1, qf[c][s][1], sc[c][t], 0, 0, 0);
                    }
            }
        }
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int t = 0; t < 4; ++t) sc[c][t] *= ks;

        if (absent || at0 < lo_most || at0 + kPage > hi_least) {
            // some row sees this page in part: masked keys count nothing, whatever their
            // bytes.  Keys that no row sees become 0; a NaN among values that some row
            // does not see (its 0 would carry it over) becomes 0 as well, and is put
            // into the rows that see it by the product of its place with what they see.
            uint32_t nan = 0;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                uint32_t keep = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = at0 + 16 * g + 4 * t + i;
                    if (!absent && j >= lo_least && j < hi_most) keep |= 0xffu << (8 * i);
#pragma unroll
                    for (int c = 0; c < NC; ++c)
                        if (absent || j < lo[c] || j >= hi[c]) sc[c][t][i] = -INFINITY;
                }
#pragma unroll
                for (int i = 0; i < VT; ++i) {
                    uint32_t& w = t == 0 ? vv[i].x : t == 1 ? vv[i].y : t == 2 ? vv[i].z : vv[i].w;
                    w &= keep;
                    nan |= nan_bytes(w);
                }
            }
            if (__any(nan != 0)) {
#pragma unroll
                for (int i = 0; i < VT; ++i) {
                    uint32_t w[4] = {vv[i].x, vv[i].y, vv[i].z, vv[i].w}, at[4];
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const uint32_t b = nan_bytes(w[t]), whole = (b >> 7) * 0xffu;
                        w[t] &= ~whole;
                        at[t] = whole & 0x38383838u;  // 1
                    }
                    vv[i] = make_uint4(w[0], w[1], w[2], w[3]);
                    const half8 v0 = e4m3x8_to_f16(at[0], at[1]), v1 = e4m3x8_to_f16(at[2], at[3]);
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        half8 s0, s1;
#pragma unroll
                        for (int t = 0; t < 4; ++t)
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int j = at0 + 16 * g + 4 * t + k;
                                const _Float16 x = (_Float16)(!absent && j >= lo[c] && j < hi[c] ? 1.f : 0.f);
                                if (t < 2) s0[4 * t + k] = x;
                                else s1[4 * (t - 2) + k] = x;
                            }
                        float4v hit = {0.f, 0.f, 0.f, 0.f};
                        hit = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, s0, hit, 0, 0, 0);
                        hit = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, s1, hit, 0, 0, 0);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (hit[k] > 0.f) o[c][i][k] = NAN;
                    }
                }
            }
        }

        half8 w_hi[NC][2], w_lo[NC][2];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (c > 0 && c >= sets) continue;
            float top = -INFINITY;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) top = fmaxf(top, sc[c][t][i]);
            top = fmaxf(top, __shfl_xor(top, 16, 64));
            top = max_across32(top);
            const bool none = top == -INFINITY;       // (the scale of a page that a row does not see does not reach it)
            const float wt = none ? wm[c] : fmaxf(wm[c], top + vs);
            top = fmaxf(top, m[c]);
            const float at = top == -INFINITY ? 0.f : top, wat = wt == -INFINITY ? 0.f : wt;
            l[c] *= __builtin_amdgcn_exp2f(m[c] - at);   // 0 from -inf
            const float fade = __builtin_amdgcn_exp2f(wm[c] - wat), by = vs + at - wat + 15.f;
            const float up = none ? 0.f : __builtin_amdgcn_exp2f(by);
            m[c] = top;
            wm[c] = wt;
#pragma unroll
            for (int i = 0; i < VT; ++i) o[c][i] *= fade;
            const bool far = __any(!none && by > 100.f);   // a weight's factor past the type: from the score itself
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = __builtin_amdgcn_exp2f(sc[c][t][i] - at);
                    l[c] += x;
                    float w = x * up;
                    if (far) w = none ? 0.f : __builtin_amdgcn_exp2f(sc[c][t][i] - wat + vs + 15.f);
                    const _Float16 a = (_Float16)w;
                    w_hi[c][t >> 1][(t & 1) * 4 + i] = a;
                    if (PARTS == 2) w_lo[c][t >> 1][(t & 1) * 4 + i] = (_Float16)(w - (float)a);
                }
        }
#pragma unroll
        for (int i = 0; i < VT; ++i) {
            const half8 v0 = e4m3x8_to_f16(vv[i].x, vv[i].y), v1 = e4m3x8_to_f16(vv[i].z, vv[i].w);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                if (c > 0 && c >= sets) continue;
                o[c][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, w_hi[c][0], o[c][i], 0, 0, 0);
                o[c][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, w_hi[c][1], o[c][i], 0, 0, 0);
                if (PARTS == 2) {
                    o[c][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, w_lo[c][0], o[c][i], 0, 0, 0);
                    o[c][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, w_lo[c][1], o[c][i], 0, 0, 0);
                }
            }
        }
    }

    // join the waves, a set at a time: sums over the lane groups, then over the waves
    const size_t heads = (size_t)p.N * p.Hq;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        if (c >= sets) break;
        l[c] += __shfl_xor(l[c], 16, 64);
        l[c] = sum_across32(l[c]);
        __syncthreads();
        if (g == 0) { s_ml[wave][col][0] = m[c]; s_ml[wave][col][1] = l[c]; }
        const float down = m[c] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(wm[c] - m[c] - 15.f);   // to the scores' maximum
#pragma unroll
        for (int i = 0; i < VT; ++i)
            *reinterpret_cast<float4v*>(&s_o[wave][col][16 * i + 4 * g]) = o[c][i] * down;
        __syncthreads();
        const int n = min(16, rows - 16 * c);
        for (int idx = threadIdx.x; idx < n * D; idx += 64 * kWaves) {
            const int cc = idx / D, ch = idx % D;
            float top = -INFINITY;
#pragma unroll
            for (int y = 0; y < kWaves; ++y) top = fmaxf(top, s_ml[y][cc][0]);
            const float at = top == -INFINITY ? 0.f : top;
            float sum = 0.f, x = 0.f;
#pragma unroll
            for (int y = 0; y < kWaves; ++y) {
                const float f = __builtin_amdgcn_exp2f(s_ml[y][cc][0] - at);
                sum += s_ml[y][cc][1] * f;
                x += s_o[y][cc][ch] * f;
            }
            const int r = row0 + 16 * c + cc;
            const size_t head = (size_t)(first + r / rep) * p.Hq + kh * rep + r % rep;
            const size_t at_row = (size_t)slot * heads + head;
            p.part_o[at_row * D + ch] = x;
            if (ch == 0) { p.part_ml[at_row * 2] = top; p.part_ml[at_row * 2 + 1] = sum; }
        }
    }
}

// Joins a head's partial results: one workgroup per head; its lanes read the maxima
// and sums side by side, then 1024 / D groups of them the outputs.
template <int D>
__global__ __launch_bounds__(256) void attn_shared_join(SharedParams p) {
    constexpr int GROUPS = 1024 / D;                  // D / 4 lanes each, four channels a lane
    __shared__ float s_x[GROUPS][D], s_ml[8], s_sum;
    const size_t head = blockIdx.x, rows = (size_t)p.N * p.Hq;
    const int tid = threadIdx.x, gi = tid / (D / 4), ch = 4 * (tid % (D / 4));
    // a sequence in no group has no shared part
    const int n = (int)(head / p.Hq), slots = p.shared_splits + p.own_splits;
    const int begin = shared_pages_of(p, n, tid & 63) > 0 ? 0 : p.shared_splits;
    float top = -INFINITY, sum = 0.f;
    for (int s = begin + tid; s < slots; s += 256) {
        const float2 ml = *reinterpret_cast<const float2*>(&p.part_ml[(s * rows + head) * 2]);
        const float both = fmaxf(top, ml.x);
        if (both != -INFINITY) sum = sum * __builtin_amdgcn_exp2f(top - both) + ml.y * __builtin_amdgcn_exp2f(ml.x - both);
        else sum += ml.y;                             // 0, or NaN where every score is
        top = both;
    }
    for (int o = 32; o > 0; o >>= 1) {
        const float t2 = __shfl_xor(top, o, 64), s2 = __shfl_xor(sum, o, 64), both = fmaxf(top, t2);
        sum = both == -INFINITY ? sum + s2
                                : sum * __builtin_amdgcn_exp2f(top - both) + s2 * __builtin_amdgcn_exp2f(t2 - both);
        top = both;
    }
    if ((tid & 63) == 0) { s_ml[2 * (tid >> 6)] = top; s_ml[2 * (tid >> 6) + 1] = sum; }
    __syncthreads();
    top = fmaxf(fmaxf(s_ml[0], s_ml[2]), fmaxf(s_ml[4], s_ml[6]));
    const float at = top == -INFINITY ? 0.f : top;
    if (tid == 0) {
        float all = 0.f;
        for (int w = 0; w < 4; ++w)
            all += top == -INFINITY ? s_ml[2 * w + 1] : s_ml[2 * w + 1] * __builtin_amdgcn_exp2f(s_ml[2 * w] - at);
        s_sum = all;
    }
    float4v x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int s = begin + gi; s < slots; s += GROUPS) {
        const float f = __builtin_amdgcn_exp2f(p.part_ml[(s * rows + head) * 2] - at);
        x += *reinterpret_cast<const float4v*>(&p.part_o[(s * rows + head) * D + ch]) * f;
    }
    *reinterpret_cast<float4v*>(&s_x[gi][ch]) = x;
    __syncthreads();
    if (tid < D) {
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) y += s_x[i][tid];
        store_out(p, head * D + tid, top == -INFINITY && !(y != y) ? 0.f : y / s_sum);
    }
}

SharedPlan attn_shared_plan(int N, int groups, int Hq, int Hkv, int max_pages, int window) {
    SharedPlan x;
    const int rep = Hq / Hkv;
    const long long rows = (long long)N * rep;        // of a key head
    x.columns = rows > 16LL * groups ? 32 : 16;
    // at most: every group's last tile is not full
    x.tiles = (int)(rows / x.columns + (groups < N ? groups : N));
    int pages = max_pages;
    if (window > 0 && window / kPage + 2 < pages) pages = window / kPage + 2;
    auto splits = [&](long long base) {
        long long s = (1024 + base - 1) / base;
        const long long most = (pages + kWaves - 1) / kWaves;
        if (s > most) s = most;
        return s < 1 ? 1 : (int)s;
    };
    x.shared_splits = splits((long long)x.tiles * Hkv);
    x.own_items = (long long)N * Hkv * ((rep + x.columns - 1) / x.columns);
    x.own_splits = splits(x.own_items);
    return x;
}

long long attn_shared_workgroups(const SharedPlan& x, int Hkv, long long heads) {
    const long long items = (long long)x.tiles * Hkv * x.shared_splits + x.own_items * x.own_splits;
    return items > heads ? items : heads;
}

template <int D> static hipError_t launch_d(const SharedParams& p, const SharedPlan& x, hipStream_t st) {
    const dim3 grid((unsigned)((long long)p.tiles * p.Hkv * p.shared_splits + x.own_items * p.own_splits)), block(64 * kWaves);
    const bool one = (p.flags & GDR_OUT_BF16) != 0;
    if (x.columns == 16) {
        if (one) hipLaunchKernelGGL((attn_shared_kernel<D, 1, 1>), grid, block, 0, st, p);
        else hipLaunchKernelGGL((attn_shared_kernel<D, 1, 2>), grid, block, 0, st, p);
    } else {
        if (one) hipLaunchKernelGGL((attn_shared_kernel<D, 2, 1>), grid, block, 0, st, p);
        else hipLaunchKernelGGL((attn_shared_kernel<D, 2, 2>), grid, block, 0, st, p);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(attn_shared_join<D>, dim3((unsigned)((long long)p.N * p.Hq)), dim3(256), 0, st, p);
    return hipGetLastError();
}

hipError_t launch_attn_shared(const SharedParams& p, const SharedPlan& x, hipStream_t st) {
    return p.d == 64 ? launch_d<64>(p, x, st) : launch_d<128>(p, x, st);
}

}  // namespace gdr
