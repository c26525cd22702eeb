"""MI355X (gfx950) DeepSeekMoE layer forward with auxiliary-loss-free routing.

The layer runs in hand-written HIP kernels behind a C ABI (include/moe.h);
this package holds those sources (csrc/), the in-tree build (build.py), the
ctypes binding (_lib.py) and a thin layer object (layer.py).
"""
from . import _lib  # noqa: F401
from ._lib import (MOE_WS_BACKWARD_SAVED, MOE_WS_ROUTER_GRAD, MOE_WS_ROUTER_LOGITS,  # noqa: F401
                   MoeError, balance_workspace_bytes, desc, ffn_weights, moe_backward, moe_backward_saved,
                   moe_balance_loss, moe_bias_update, moe_checkpoint_pack, moe_checkpoint_unpack, moe_combine,
                   moe_combine_backward, moe_dispatch, moe_expert_down, moe_expert_ffn, moe_expert_gate_up,
                   moe_expert_gate_up_rows, moe_route, moe_router_logits, moe_router_logits_backward, moe_select,
                   moe_select_backward, saved, selection, workspace_bytes)
