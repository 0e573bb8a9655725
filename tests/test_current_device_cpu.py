"""No GPU: arguments on another device than the current one are refused before
anything is allocated or launched.  The library launches on the current device,
and a default stream's handle says nothing of the device it belongs to."""
import pytest
import torch

import linear_attention_sequence_device_gb300 as g
from linear_attention_sequence_device_gb300 import binding, ssm


class Elsewhere:
    """What the front end may ask of a tensor on device 1 before it refuses it; anything else fails the test."""
    dtype = torch.bfloat16
    is_cuda = True

    def get_device(self):
        return 1


@pytest.fixture(autouse=True)
def device_0(monkeypatch):
    monkeypatch.setattr(binding, "_current_device", lambda: 0)

    def used(*a, **kw):
        raise AssertionError("allocated or launched")
    for name in ("empty", "empty_like"):
        monkeypatch.setattr(torch, name, used)
    monkeypatch.setattr(ssm, "_run", used)
    monkeypatch.setattr(ssm, "_raw_stream", used)


X = Elsewhere()
CALLS = dict(conv_fwd=lambda: g.gdn_ssm_conv_fwd(X, X, X, X), conv_bwd=lambda: g.gdn_ssm_conv_bwd(X, X, X, X, X),
             conv_step=lambda: g.gdn_ssm_conv_step(X, X, X, X), scan_fwd=lambda: g.gdn_ssm_scan_fwd(X, X, X, X, X, X),
             scan_bwd=lambda: g.gdn_ssm_scan_bwd(X, X, X, X, X, X, X, X),
             scan_step=lambda: g.gdn_ssm_scan_step(X, X, X, X, X, X), norm_fwd=lambda: g.gdn_block_norm_fwd(X, X, X),
             norm_bwd=lambda: g.gdn_block_norm_bwd(X, X, X, X, X))


@pytest.mark.parametrize("name", CALLS)
def test_scan_layer_and_block_norm(name):
    with pytest.raises(ValueError, match="current device"):
        CALLS[name]()


def test_on_the_current_device(monkeypatch):
    monkeypatch.setattr(binding, "_current_device", lambda: 1)
    assert ssm._lead(X, "x") == (1, binding.GDN_BF16)


LAYER = dict(chunk_fwd=lambda: g.gdn_chunk_fwd(X, X, X, X, X, X), chunk_bwd=lambda: g.gdn_chunk_bwd(X, X, X, X, X, X, X),
             chunk_heads=lambda: binding.gdn_chunk_fwd_heads(X, X, X, X, X, X),
             summary=lambda: g.gdn_chunk_summary(X, X, X, X, X), conv=lambda: g.gdn_conv_silu(X, X, None, X),
             plan=lambda: g.gdn_cp_plan(X, 2), combine=lambda: g.gdn_state_combine(X, X),
             shard=lambda: g.gdn_shard_fwd(X, X, None, X, X, X, 1, 1, 32, 32, 2),
             noalloc=lambda: binding.gdn_shard_fwd_noalloc(X, X, None, X, X, X, 1, 1, 32, 32, 2),
             layer=lambda: g.gdn_layer_fwd(X, X, None, X, X, X, X, X, X, X, 1, 1, 32, 32, 2),
             head_major=lambda: binding.to_head_major(X), token_major=lambda: binding.to_token_major(X))


@pytest.mark.parametrize("name", LAYER)
def test_gated_delta_net_layer(name, monkeypatch):
    # the first argument of most is of the element type, of two of another
    monkeypatch.setattr(Elsewhere, "dtype", dict(plan=torch.int32, combine=torch.float32).get(name, torch.bfloat16))
    with pytest.raises(ValueError, match="current device"):
        LAYER[name]()
