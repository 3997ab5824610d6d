"""What the Python calls around the indexer hand to the library, on the CPU: host tensors stand
for device ones, and the library's call is recorded instead of made."""

import types

import pytest
import torch

import mxfp4_paged_cache_quant_amd as mx


@pytest.fixture
def calls(monkeypatch):
    made = []
    monkeypatch.setattr(mx, "_device_of", lambda t, name: types.SimpleNamespace(index=-1))
    monkeypatch.setattr(mx, "_call", lambda name, device, stream, *args: made.append((name, args)))
    return made


def _attn(**change):
    args = dict(q=torch.zeros((2, 4, 192), dtype=torch.bfloat16),
                cache=torch.zeros((3, 64, 192), dtype=torch.bfloat16),
                block_table=torch.zeros((2, 40), dtype=torch.int32), ke=torch.ones(2, dtype=torch.int32), scale=0.1,
                out=torch.zeros((2, 4, 128), dtype=torch.bfloat16), lse=torch.zeros((2, 4)))
    return mx.attn_paged(**{**args, **change})


def test_attn_hands_over_a_whole_workspace(calls):
    ws = torch.zeros(4096, dtype=torch.uint8)
    _attn(workspace=ws)
    assert calls[0][0] == "idx_attn_paged" and calls[0][1][-2:] == (ws.data_ptr(), 4096)


@pytest.mark.parametrize("workspace", [
    torch.zeros(256, dtype=torch.uint8).expand(1 << 20, 256),     # 256 bytes that look like many
    torch.zeros(1, dtype=torch.uint8).expand(1 << 28), torch.zeros(8192, dtype=torch.uint8)[::2]])
def test_attn_refuses_a_workspace_whose_size_is_not_its_memory(calls, workspace):
    with pytest.raises(mx.MxidxError, match="workspace must be contiguous"):
        _attn(workspace=workspace)
    assert not calls
