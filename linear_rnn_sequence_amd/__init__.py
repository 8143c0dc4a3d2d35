"""MI355X (gfx950) WKV7 recurrence of RWKV-7 and gated delta rule: hand-written HIP kernels
behind a C ABI (include/rwkv7_wkv.h, include/gated_delta.h), with this package as its Python
binding."""
from .gated_delta import (STATE_MOVE_MAX, gated_delta_backward,  # noqa: F401
                          gated_delta_backward_workspace_bytes, gated_delta_chunks,
                          gated_delta_ckpt_size, gated_delta_decode, gated_delta_forward,
                          gated_delta_forward_train, gated_delta_forward_workspace_bytes,
                          state_move)
from .wkv import (ALGOS, CKPT_INTERVAL, Rwkv7Error, abi_version, backward,  # noqa: F401
                  backward_workspace_bytes,
                  decode, decode_fused, forward, forward_bidir, forward_bidir_workspace_bytes,
                  forward_fused, forward_noalloc, forward_train,
                  forward_workspace_bytes, lib, prepare_decode, stream_copy)
