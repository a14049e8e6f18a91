#include "stream.h"
namespace saf3r {
size_t attn_workspace_bytes(int n_seqs, int n_tokens, int n_heads) { return 256; }
saf3r_status launch_attn(const KvAttnParams& p, cudaStream_t stream, int* n_launch) { return SAF3R_ERR_UNSUPPORTED; }
}
