// Internal interface of the kernels for several continuations of one prompt
// (gdr_shared.hip, gdr_pages.hip, gdr_beam.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/gdr.h"

namespace gdr {

// The paged cache and its tables, as gdr_kv_fork and gdr_kv_compact change them.
struct PagesParams {
    uint8_t* k_cache;
    uint8_t* v_cache;
    float* k_scale;
    float* v_scale;
    const int* block_table;     // [N_in, max_pages]
    const int* cache_len;       // [N_in]
    const int* parent;          // [N], or null: row n
    const int* room;            // [N], or null: room_all
    const uint8_t* held;        // [n_pages], or null
    int* table_out;             // [N, max_pages]
    int* len_out;               // [N] (fork)
    int* missing;               // [N] (fork)
    int* used;                  // [1] (compact)
    int N_in, N, room_all, Hkv, d, n_pages, max_pages;
    void* workspace;
};
size_t kv_fork_workspace(int N, int n_pages);
size_t kv_compact_workspace(int n_pages);
// Workgroups of a call's largest launch.
long long kv_fork_workgroups(int N, int Hkv, int d, int n_pages, int max_pages);
long long kv_compact_workgroups(int N, int n_pages, int max_pages);
hipError_t launch_kv_fork(const PagesParams& p, hipStream_t st);
hipError_t launch_kv_compact(const PagesParams& p, hipStream_t st);

// How a call of attention over shared pages is dealt out, from what the host knows, and
// where the parts of its workspace start.
struct SharedPlan {
    int width;                  // rows of a workgroup for shared pages: 32 or 64
    long long units;            // (group, key head, `width` of its rows) that there can be
    int workgroups;             // for the shared pages, at most
    bool few;                   // groups and sequences: no plan kernel
    long long own_items;        // (sequence, key head, set of 16 query heads)
    int own_splits;             // runs that a sequence's own pages are dealt into
    size_t at_head, at_groups, at_sequences, at_items, at_part_o, at_part_ml, at_own_o, at_own_ml, bytes;
};
constexpr int kMostGroups = 4096;                     // the plan has them in LDS
struct SharedParams {
    const void* q;
    const uint8_t* k_cache;
    const uint8_t* v_cache;
    const float* k_scale;
    const float* v_scale;
    const int* block_table;
    const int* cache_len;
    const int* group_start;     // [groups + 1]
    const int* shared_pages;    // [groups]
    void* o;
    void* plan_head;            // workgroups, pages of each
    void* plan_groups;          // [groups]
    void* plan_sequences;       // [N] each sequence's group, as in plan_groups
    int* plan_items;            // [workgroups] the group that one starts in
    float* part_o;              // [units + workgroups, width, d] unnormalised
    float* part_ml;             // [units + workgroups, width, 2] maximum (base 2) and sum
    float* own_o;               // [own_splits, N, Hq, d] and its maxima and sums
    float* own_ml;
    int N, groups, Hq, Hkv, d, n_pages, max_pages, window;
    int width, units, workgroups, own_splits, few;
    long long own_runs;         // own_items * own_splits
    float scale;
    uint32_t flags;
};
SharedPlan attn_shared_plan(int N, int groups, int Hq, int Hkv, int d, int max_pages, int window);
long long attn_shared_workgroups(const SharedPlan& x, long long heads);
hipError_t launch_attn_shared(const SharedParams& p, hipStream_t st);

constexpr int kMostBeams = 64, kMostSelected = 64;
constexpr int kMostTokens = 1 << 26;                  // of a vocabulary
struct BeamParams {
    const void* logits;         // [G * K] rows of V, `stride` elements apart
    const float* scores;        // [G * K]
    const uint8_t* ended;       // [G * K], or null
    int* tokens;                // [G, M]
    int* rows;                  // [G, M]
    float* scores_out;          // [G, M]
    uint8_t* ended_out;         // [G, M]
    int G, K, M, V, end_token;
    long long stride;
    uint32_t flags;
    int segs;                   // workgroups of a row
    uint64_t* best;             // workspace [G * K, segs, M]: the segments' best, 0 where there is none
    float* part;                // workspace [G * K, segs, 2]: their maxima and sums
};
int beam_segments(int G, int K, int V);
hipError_t launch_beam_select(const BeamParams& p, hipStream_t st);

struct ReorderParams {
    uint8_t* state;             // [layers, N, row_bytes]
    const int* parent;          // [N]
    int layers, N, K;
    long long row_bytes;
};
long long state_reorder_workgroups(int layers, int N, int K, long long row_bytes);
hipError_t launch_state_reorder(const ReorderParams& p, hipStream_t st);

}  // namespace gdr
