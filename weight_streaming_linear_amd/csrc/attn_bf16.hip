// attn_decode over a bf16 cache.
#include "attn_kernel.h"

namespace wsl {
template int launch_attn_fmt<WSL_KV_BF16>(AttnArgs &, int, hipStream_t);
}  // namespace wsl
