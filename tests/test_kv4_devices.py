"""Calls whose tensors, workspace, stream and current device are not one: refused before anything is
launched.  (Devices are stood in for: no GPU is needed.)"""
import types

import pytest
import torch


@pytest.fixture
def api(monkeypatch):
    import speculative_decoding_verify_09_gb300 as pkg
    pkg.build()
    api = pkg.load()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    return api


def on(device):
    """Arguments, a workspace and a stream on a device."""
    args = api_args()
    args._device = device
    ws = types.SimpleNamespace(buf=types.SimpleNamespace(device=torch.device("cuda", device)), ptr=256, nbytes=1 << 20)
    return args, ws, types.SimpleNamespace(device_index=device, cuda_stream=0)


def api_args():
    from speculative_decoding_verify_09_gb300 import _binding
    return _binding.Kv4AttnArgs()           # (of no shape: the library refuses it, too)


def test_a_workspace_of_another_device(api):
    args, _, stream = on(0)
    for kw in ({}, {"stream": stream}):
        with pytest.raises(ValueError, match="workspace on cuda:1"):
            api.spec_kv4_attn(args, on(1)[1], **kw)


def test_another_current_device(api):
    args, ws, _ = on(1)
    with pytest.raises(ValueError, match="current device"):
        api.spec_kv4_attn(args, ws)
    with pytest.raises(ValueError, match="current device"):
        api.kv4_workspace(args)


def test_a_stream_of_another_device(api):
    args, ws, _ = on(0)
    with pytest.raises(ValueError, match="stream on cuda:1"):
        api.spec_kv4_attn(args, ws, stream=on(1)[2])


def test_one_device_reaches_the_library(api):
    args, ws, stream = on(0)
    with pytest.raises(Exception, match="kv4_attn: "):
        api.spec_kv4_attn(args, ws, stream=stream)
