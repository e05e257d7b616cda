// Internal host interface of the 4-bit cache's kernels (beside pa_launch.h, whose argument structs they
// take: k_cache, and for the fused step k_store, is the cache).
#pragma once

#include "pa_launch.h"

namespace pa {

constexpr int kInt4ReadWarps = 2;   // of a CTA that reads rows back, a record each

// Rows of sequences read back: row_start[s] + i of k_out and v_out is token first[s] + i.
struct ReadInt4Args {
  const uint8_t* cache;             // [num_blocks][Hkv][PA_INT4_RECORD_BYTES]
  const int32_t* row_start;         // [S + 1]
  const int32_t* first;             // [S], or null: 0
  const int32_t* block_tables;      // [S][max_blocks]
  __nv_bfloat16* k_out;             // [num_rows][Hkv][128]
  __nv_bfloat16* v_out;
  int num_seqs, num_rows, max_rows, num_kv_heads, num_blocks, max_blocks;
  unsigned* status;
};

cudaError_t launch_rope_int4_store(const RopeFormArgs& a, cudaStream_t stream);
cudaError_t launch_read_int4(const ReadInt4Args& a, cudaStream_t stream);
cudaError_t launch_decode_int4(const DecodeArgs& a, cudaStream_t stream);
cudaError_t launch_prefill_int4(const PrefillArgs& a, cudaStream_t stream);
// {max_ns, seed} of its roles' sleeps (pa_set_timing_jitter).
cudaError_t set_prefill_int4_jitter(const uint32_t (&hook)[2]);

// The merge of the pieces of split sequences (paged_decode_block.cu): partial rows in a.ws_o, their (shift, sum)
// in a.ws_ml, cut as by a.num_warps warps.  `cfg` has the stream and the attributes.
cudaError_t launch_block_merge(const DecodeArgs& a, cudaLaunchConfig_t cfg);

}  // namespace pa
