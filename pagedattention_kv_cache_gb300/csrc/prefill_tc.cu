// The plain tcgen05 prefill (prefill_tc.cuh), its split rule and workspace size.
#include "prefill_tc.cuh"

namespace pkv {

// Parts a long pair may run as when the pairs alone leave SMs idle: as many
// as fit in one wave of one CTA per SM (at most kMaxParts), so the split
// never adds a second, mostly empty wave; 1 when the pairs fill the GPU.
int prefill_tc_parts(int batch, int num_kv_heads, int group, int max_seqlen_q, int sms) {
  const long long tq = kBM / group;
  const long long pairs = static_cast<long long>(batch) * num_kv_heads * ((max_seqlen_q + 2 * tq - 1) / (2 * tq));
  if (pairs <= 0 || 2 * pairs > sms) return 1;
  return static_cast<int>(std::min<long long>(kMaxParts, sms / pairs));
}

// Bytes of each of the two int arrays (tickets, ready counts) at the start of
// the prefill workspace: a half of the fixed counter area (split launches have
// at most one item per SM, far below its 8,192 counters), more only past it.
size_t prefill_tc_flag_bytes(long long items) {
  return std::max(kWorkspaceCounterBytes / 2, static_cast<size_t>((items * 4 + 255) / 256 * 256));
}

// Workspace of the tcgen05 prefill: tickets and ready counts (the counter
// area), then P records per (sequence, KV head, query tile); 0 when the
// current device's SMs are filled without splitting.
size_t prefill_tc_workspace_bytes(int batch, int num_kv_heads, int group, int head_dim, int max_seqlen_q) {
  if (batch <= 0 || num_kv_heads <= 0 || max_seqlen_q <= 0) return 0;
  if (head_dim != 64 && head_dim != 128) return 0;
  if (group != 1 && group != 2 && group != 4 && group != 8) return 0;
  DeviceInfo info;
  if (device_info(&info) != PKV_OK) return 0;
  const int parts = prefill_tc_parts(batch, num_kv_heads, group, max_seqlen_q, info.sms);
  if (parts == 1) return 0;
  const long long tq = kBM / group;
  const long long items = static_cast<long long>(batch) * num_kv_heads * 2 * ((max_seqlen_q + 2 * tq - 1) / (2 * tq));
  const size_t flags = prefill_tc_flag_bytes(items);
  const size_t record = head_dim == 64 ? Geo<64>::kRecordBytes : Geo<128>::kRecordBytes;
  return 2 * flags + static_cast<size_t>(items) * parts * record;
}

bool prefill_tc_supported(const PrefillArgs& a) {
  if (a.group != 1 && a.group != 2 && a.group != 4 && a.group != 8) return false;
  if (a.head_dim != 64 && a.head_dim != 128) return false;
  if (a.total_q <= 0) return false;
  if (a.block_tables) {
    const int bs = a.block_size;
    const bool whole_tiles = bs % kBN == 0;
    const bool pieces = bs >= 8 && kBN % bs == 0;
    if (!(whole_tiles || pieces)) return false;
    if (static_cast<long long>(a.num_blocks) * bs <= 0) return false;
  } else if (a.total_k <= 0) {
    return false;
  }
  return true;
}

int prefill_tc_launch(const PrefillArgs& a, cudaStream_t stream) { return launch_form<kPlain>(a, stream); }

}  // namespace pkv
