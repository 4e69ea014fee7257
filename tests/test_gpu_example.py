"""The serving example, its attention checked against the oracle over the
codes that its own cache holds."""
import importlib.util
import os

import numpy as np
import pytest

import oracle
from test_gpu_attention import check, limit

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_paged_serving_example():
    spec = importlib.util.spec_from_file_location(
        "paged_serving", os.path.join(ROOT, "examples", "paged_serving.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    steps = 0
    for layer, new, cached, y, q, o in example.serve(
            prompts=(70, 5, 130, 33), chunk=64, decode_steps=3, hidden=256, heads=10, kv_heads=2,
            d=64, page_size=16):
        print("[gpu-example] step", steps, new, cached, flush=True)
        assert bool(y.isfinite().all())
        scales = [np.float32(s.cpu().numpy()[0]) for s in (layer.k_scale, layer.v_scale)]
        table = layer.table.cpu().numpy()
        at, want, bound = 0, [], []
        for r, (n, c) in enumerate(zip(new, cached)):
            ids = table[r, :-(-(n + c) // 16)]
            assert (ids >= 0).all()
            k, v = (oracle.kv_decode(cache.cpu().numpy()[ids], s).transpose(0, 2, 1, 3).reshape(
                -1, 2, 64)[:n + c] for cache, s in zip((layer.k_cache, layer.v_cache), scales))
            got = oracle.attention(q[at:at + n].double().cpu().numpy(), k, v, 0.125)
            want.append(got[0])
            bound.append(limit(*got, 64, n + c, True))
            at += n
        check(o, (np.concatenate(want), np.concatenate(bound)), steps)
        # no page is held twice
        held = table[table >= 0]
        assert len(set(held.tolist())) == len(held)
        steps += 1
    assert steps >= 5
