"""Sizes past the library's limits are refused by the binding: the library takes
them as C ints, and 2^32 + 4 rows must not become 4."""
import pytest
import torch

MANY = (1 << 32) + 4


def _meta(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")


def _f32(*shape):
    return _meta(*shape, dtype=torch.float32)


CALLS = {
    "layernorm_fwd rows": lambda jg: jg.layernorm_fwd(_meta(MANY, 8), _f32(8), _f32(8), 1e-6),
    "layernorm_fwd leading dims": lambda jg: jg.layernorm_fwd(_meta(1 << 16, (1 << 16) + 1, 8), _f32(8), _f32(8), 1e-6),
    "layernorm_fwd dim": lambda jg: jg.layernorm_fwd(_meta(2, MANY), _f32(MANY), _f32(MANY), 1e-6),
    "layernorm_bwd rows": lambda jg: jg.layernorm_bwd(_meta(MANY, 8), _meta(MANY, 8), _f32(8), _f32(MANY), _f32(MANY)),
    "linear_ce_fwd rows": lambda jg: jg.linear_ce_fwd(_meta(MANY, 8), _meta(4, 8), None, _meta(MANY, dtype=torch.int64)),
    "linear_ce_fwd classes": lambda jg: jg.linear_ce_fwd(_meta(4, 8), _meta(MANY, 8), None, _meta(4, dtype=torch.int64)),
    "linear_ce_fwd width": lambda jg: jg.linear_ce_fwd(_meta(4, MANY), _meta(4, MANY), None, _meta(4, dtype=torch.int64)),
    "linear_ce_bwd rows": lambda jg: jg.linear_ce_bwd(1.0, _meta(MANY, 8), _meta(4, 8), None,
                                                      _meta(MANY, dtype=torch.int64), _f32(MANY)),
    "gated_ffn_fwd rows": lambda jg: jg.gated_ffn_fwd(_meta(MANY, 8), _meta(4, 8), _meta(4, 8)),
    "gated_ffn_bwd hidden": lambda jg: jg.gated_ffn_bwd(_meta(2, MANY), _meta(2, 8), _meta(MANY, 8), _meta(MANY, 8)),
    "linear_bwd rows": lambda jg: jg.linear_bwd(_meta(MANY, 4), _meta(MANY, 8), _meta(4, 8)),
    "linear_bwd outputs": lambda jg: jg.linear_bwd(_meta(2, MANY), _meta(2, 8), _meta(MANY, 8)),
    "one past the limit": lambda jg: jg.gated_ffn_fwd(_meta((1 << 24) + 1, 8), _meta(4, 8), _meta(4, 8)),
}


@pytest.mark.parametrize("call", CALLS)
def test_refused(call):
    import video_vit_encoder_gb300 as jg
    with pytest.raises(ValueError, match="at most 16777216 rows and columns"):
        CALLS[call](jg)


def test_the_limit_itself_is_not_refused():
    """The next check is the device's."""
    import video_vit_encoder_gb300 as jg
    with pytest.raises(ValueError, match="CUDA device"):
        jg.layernorm_fwd(_meta(1 << 24, 8), _f32(8), _f32(8), 1e-6)
    with pytest.raises(ValueError, match="CUDA device"):
        jg.gated_ffn_fwd(_meta(1 << 24, 8), _meta(4, 8), _meta(4, 8))
