// Sort of tokens by the row that they point to (sort.cu), as the sums over sorted
// tokens use it (sums.cuh).
#pragma once

#include "rows.h"

namespace mk {

constexpr uint32_t kNone = 0xFFFFFFFFu;     // no row: above every table's last one

// Factors of a CP model as tables in shared memory: neighbouring modes form groups,
// and a group's table has the products of its modes' rows, one for every combination
// of their indices (the last mode's fastest).
constexpr int kMaxGroups = MTTKRP_MAX_ORDER;
constexpr int kFewGroups = 4;

struct Tables {
    int groups;
    int rows;                               // of all groups
    struct Group {
        int modes;
        int mode[MTTKRP_MAX_ORDER];
        int first;                          // the group's first row
    } group[kMaxGroups];
};

// Sorted tokens: d lists of n entries of `bytes` bytes, which begin with the row
// (kNone, behind all others, for tokens that take no part).  8 bytes: the token
// follows.  16 or 32 bytes: g of the token, then its row in the table of each group of
// `tables` as 16-bit numbers, kFewGroups or kMaxGroups of them.
struct Sorted {
    const char* entries;
    int bytes;
};

struct SortPlan {
    int passes, bits, bins, ctas, items;
    int64_t per_cta;
    int entry_bytes;
    size_t pairs, counts;                   // bytes of one buffer of entries, and of the counts
    size_t total() const { return 2 * pairs + counts; }
};

// The sort's CTAs wait for one another, so there are at most `sms` of them: kSms for the
// workspace, which fewer never outgrow, sort_sms() for a launch.
SortPlan plan_sort(const IndexArgs& index, int entry_bytes, int sms);
// SMs of the current device, at most kSms
int sort_sms();
// tables: nullptr, or one for each index column, for entries of 16 or 32 bytes
cudaError_t sort_tokens(const IndexArgs& index, const SortPlan& p, void* ws, const Tables* tables, const float* g,
                        Sorted& sorted, cudaStream_t s);
// one index column of at most 16384 tokens, by one cluster of CTAs while the others set `bytes` bytes at `out`
// (16-byte aligned) to zero
cudaError_t sort_and_fill(const IndexArgs& index, const SortPlan& p, void* ws, void* out, int64_t bytes,
                          Sorted& sorted, cudaStream_t s);

}  // namespace mk
