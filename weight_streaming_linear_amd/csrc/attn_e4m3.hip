// attn_decode over an e4m3 cache.
#include "attn_kernel.h"

namespace wsl {
template int launch_attn_fmt<WSL_KV_E4M3>(AttnArgs &, int, hipStream_t);
}  // namespace wsl
