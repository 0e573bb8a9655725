"""Context-parallel Gated DeltaNet forward for one GB300 (sm_103a).

The computation lives in the CUDA library ``libgdncp.so`` (C ABI declared in
``include/gdn_cp.h``); ``binding`` is its thin Python front end.
"""
from .binding import (GdnError, decode_plan, gdn_chunk_fwd, gdn_chunk_summary,  # noqa: F401
                      gdn_conv_silu, gdn_cp_plan, gdn_layer_fwd, gdn_shard_fwd, gdn_state_combine, load,
                      plan_words, shard_fwd_workspace_size, shard_fwd_workspace_min_size)
from .binding import chunk_bwd_workspace_size, gdn_chunk_bwd  # noqa: F401
from .ssm import (gdn_block_norm_bwd, gdn_block_norm_fwd, gdn_ssm_conv_bwd, gdn_ssm_conv_fwd,  # noqa: F401
                  gdn_ssm_conv_step, gdn_ssm_scan_bwd, gdn_ssm_scan_fwd, gdn_ssm_scan_step,
                  ssm_scan_bwd_workspace_size, ssm_scan_ckpt_shape, ssm_scan_workspace_size)
from .lm import (embed_bwd_workspace_size, gdn_chunk_step, gdn_embed_bwd, gdn_embed_fwd, gdn_layer_step,  # noqa: F401
                 gdn_vocab_loss_bwd, gdn_vocab_loss_fwd, vocab_loss_bwd_workspace_size, vocab_loss_fwd_workspace_size)
