// Internal launch interface of the operators for sequences that share pages of
// one cache.
#pragma once

#include "tokens.h"

namespace prhs {

// What a row of the batch becomes: columns [0, keep) of row `from`, new pages up
// to column `blocks`, nothing up to column `held`; columns [released, held) of its
// old row give their pages back.
struct __align__(16) PageRow {
  int from, keep, blocks, released, held;
  int len;    // new length; -1: the row stays as it is
  int taken;  // new pages of the rows before it
  int last;   // (fork) the page whose rows go to the new page; -1: none
};

struct PagesLaunch {
  KVView kv;              // block_table and seq_lens: the state before
  const int32_t* n_pages;
  const int32_t* shares;
  const int32_t* free_pages;
  const int32_t* free_head;
  int n_free;
  int32_t* table_out;
  int32_t* lens_out;
  int32_t* n_pages_out;
  int32_t* shares_out;
  int32_t* free_out;
  int32_t* head_out;
  const int32_t* parent;  // fork; null: compact
  const int32_t* keep;    // compact: [B][cap]
  const int32_t* keep_n;
  int cap;                // columns of src and dst (fork: block_size)
  int32_t* src;
  int32_t* dst;
  // workspace
  PageRow* rows;   // [B]
  int32_t* stage;  // [B][max_blocks]: the new rows of the table, until the old ones are read
  int2* part;      // [B][chunks of kept positions]: (positions kept in place, error bits)
  int* sums;       // [warps of the launch] pages given back, then one word of error bits
};
size_t pages_workspace(const KVView& kv);
void pages_split(PagesLaunch* a, void* ws);
cudaError_t launch_pages(const PagesLaunch& a, int sms, cudaStream_t s);

struct CopyLaunch {
  KVView to, from;
  int n;
  const int32_t* src;
  const int32_t* dst;
};
cudaError_t launch_copy_rows(const CopyLaunch& a, cudaStream_t s);

struct FindLaunch {
  KVView kv;
  const int32_t* cu_new;
  int min_keys;
  int4* shared;
};
cudaError_t launch_find_shared(const FindLaunch& a, cudaStream_t s);

}  // namespace prhs
