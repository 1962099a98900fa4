"""GB300 (sm_103a) V-JEPA 2 / 2.1 video ViT encoder forward, and operators for
training a classifier, gated MLP blocks and a recurrent decoder on its tokens.

The compute lives in ``libjepa_gb300.so`` (hand-written CUDA behind the C ABI
of ``include/jepa_gb300.h``); this package only marshals arguments.
"""
from ._lib import JepaError, LIB_PATH, load  # noqa: F401
from .binding import (  # noqa: F401
    Encoder, Head, Predictor, attention, blob_check, encoder_params, encoder_tensor_order, head_params, head_tensor_order,
    layernorm_f32, linear,
    ops_sync, pack_blob, predictor_params, predictor_tensor_order, qkv_rope, rope3d_f32,
    selftest_scan_wait_timeout, selftest_wait_timeout,
)
from .decoder import (  # noqa: F401
    embedding_bwd, embedding_fwd, gated_scan_bwd, gated_scan_fwd, linear_distill_bwd, linear_distill_fwd,
)
from .training import (  # noqa: F401
    gated_ffn_bwd, gated_ffn_fwd, layernorm_bwd, layernorm_fwd, linear_bwd, linear_ce_bwd, linear_ce_fwd,
)
