"""The decoder-layer example's workspaces, on the CPU: one that a captured step may use is never freed."""
import importlib.util
import os
import weakref

import torch

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_layer.py")


def test_replaced_workspaces_stay_allocated():
    spec = importlib.util.spec_from_file_location("decoder_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    layer = m.Layer.__new__(m.Layer)
    layer.w_out, layer.workspaces = torch.empty(1), {}
    small = layer.workspace("attention", 100)
    ref, address = weakref.ref(small), small.data_ptr()
    assert layer.workspace("attention", 60).data_ptr() == address     # the same one serves smaller calls
    del small
    large = layer.workspace("attention", 200)
    assert large.numel() >= 200 and not large.any()
    assert ref() is not None and layer.workspace("attention", 100).data_ptr() == large.data_ptr()
