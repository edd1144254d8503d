// Arguments of the attention kernels (internal).
#pragma once

#include "kv_common.h"

namespace skg {

struct TreeArgs {
  KvView cache;
  const uint8_t* q;
  int64_t ldq;  // bytes
  uint8_t* o;   // or null
  int64_t ldo;  // bytes
  uint8_t* oq;  // or null
  const int32_t* cu;  // or null: n_tokens / n_seqs each
  const int32_t* ctx;
  const int32_t* table;
  int64_t width;
  int64_t max_kv;
  const uint64_t* mask;  // or null: a chain
  float scale;
  int64_t T;
  int n_seqs;
  int hq;
  int group;  // query heads of a cache head
  int max_draft;
};

}  // namespace skg
