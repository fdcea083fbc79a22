"""Tree attention, read-back and rotary positions without a GPU: the frequencies, the
workspace size and every refusal on the host."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

import quantised_kv_cache_kvq_gb300 as K
from quantised_kv_cache_kvq_gb300 import _native as N

P = 0x10000          # an aligned address that no refused call reads


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def rope_config(**kw):
    base = dict(head_dim=128, rotary_dim=128, layout=0, dtype=0, scaling=0, original_context=8192, base=10000.0,
                factor=8.0, low=1.0, high=4.0, magnitude=1.0)
    base.update(kw)
    return K.KvqRopeConfig(**base)


def frequencies64(base, R, scaling, factor, low, high, original):
    i = np.arange(R // 2)
    b = base * factor ** (R / (R - 2)) if scaling == 2 else base
    w = b ** (-2.0 * i / R)
    if scaling == 1:
        w = w / factor
    if scaling == 3:
        turns = original * w / (2 * np.pi)
        for j in range(R // 2):
            if turns[j] <= low:
                w[j] /= factor
            elif turns[j] < high:
                g = (turns[j] - low) / (high - low)
                w[j] = g * w[j] + (1 - g) * w[j] / factor
    return w


@pytest.mark.parametrize("scaling", [0, 1, 2, 3])
@pytest.mark.parametrize("base,R,factor,low,high,original", [
    (10000.0, 128, 8.0, 1.0, 4.0, 8192), (500000.0, 64, 16.0, 1.0, 32.0, 4096), (10000.0, 4, 2.0, 0.5, 1.0, 1),
    (10000.0, 256, 1.0, 1.0, 4.0, 2048)])
def test_frequencies_follow_their_formula(scaling, base, R, factor, low, high, original):
    w = np.array(K.kvq_rope_frequencies(rope_config(head_dim=256, rotary_dim=R, scaling=scaling, base=base,
                                                    factor=factor, low=low, high=high, original_context=original)))
    # one rounding to binary32 of a binary64 value a few of its own steps off
    np.testing.assert_allclose(w, frequencies64(base, R, scaling, factor, low, high, original), rtol=2.0 ** -24 + 1e-14)


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=3), dict(rotary_dim=130), dict(head_dim=512, rotary_dim=258), dict(head_dim=0),
    dict(head_dim=1025), dict(layout=2), dict(layout=-1), dict(dtype=2), dict(scaling=4), dict(scaling=-1),
    dict(base=0.0), dict(base=-1.0), dict(base=math.inf), dict(base=math.nan), dict(scaling=1, factor=0.0),
    dict(scaling=2, factor=math.nan), dict(scaling=2, rotary_dim=2), dict(scaling=3, high=1.0),
    dict(scaling=3, low=math.nan), dict(scaling=3, original_context=0)])
def test_frequencies_refuse(kw):
    with pytest.raises(K.KvqError) as e:
        K.kvq_rope_frequencies(rope_config(**kw))
    assert e.value.code == N.KVQ_ERR_ARG


def rope(**kw):
    a = dict(rope=rope_config(), w=(C.c_float * 64)(), positions=P, tokens=4, q=P, q_out=P + 65536, q_heads=2,
             q_stride=256, q_out_stride=256, k=P, k_out=P + 131072, kv_heads=1, k_stride=128, k_out_stride=128, flags=0,
             stream=0)
    a.update(kw)
    return K.kvq_rope(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(w=None), N.KVQ_ERR_ARG), (dict(positions=None), N.KVQ_ERR_ARG), (dict(q=None), N.KVQ_ERR_ARG),
    (dict(q_out=None), N.KVQ_ERR_ARG), (dict(k=None), N.KVQ_ERR_ARG), (dict(k_out=None), N.KVQ_ERR_ARG),
    (dict(tokens=-1), N.KVQ_ERR_ARG), (dict(tokens=1 << 31), N.KVQ_ERR_ARG), (dict(q_heads=-1), N.KVQ_ERR_ARG),
    (dict(kv_heads=-1), N.KVQ_ERR_ARG), (dict(flags=2), N.KVQ_ERR_ARG), (dict(q_stride=255), N.KVQ_ERR_ARG),
    (dict(q_out_stride=128), N.KVQ_ERR_ARG), (dict(k_stride=0), N.KVQ_ERR_ARG),
    (dict(q_out=P, q_out_stride=512), N.KVQ_ERR_ARG), (dict(q=P + 1), N.KVQ_ERR_ALIGN), (dict(k_out=P + 1), N.KVQ_ERR_ALIGN),
    (dict(positions=P + 2), N.KVQ_ERR_ALIGN), (dict(rope=rope_config(rotary_dim=7)), N.KVQ_ERR_ARG)])
def test_rope_refuses(kw, code):
    with pytest.raises(K.KvqError) as e:
        rope(**kw)
    assert e.value.code == code


def test_rope_with_nothing_to_do():
    rope(tokens=0, positions=None, q=None, q_out=None, k=None, k_out=None)
    rope(q_heads=0, kv_heads=0, q=None, q_out=None, k=None, k_out=None)


def config(**kw):
    base = dict(scheme=0, layers=2, batch=3, q_heads=8, kv_heads=2, head_dim=128, bits=2, group_k=32, group_v=32,
                residual=64, max_tokens=512, in_dtype=0)
    base.update(kw)
    return K.KvqConfig(**base)


@pytest.mark.parametrize("kw,call,code", [
    (dict(bits=3), {}, N.KVQ_ERR_ARG), (dict(scheme=7), {}, N.KVQ_ERR_ARG), ({}, dict(cache=None), N.KVQ_ERR_ARG),
    ({}, dict(layer=2), N.KVQ_ERR_ARG), ({}, dict(layer=-1), N.KVQ_ERR_ARG), ({}, dict(seq_begin=-1), N.KVQ_ERR_ARG),
    ({}, dict(seq_begin=1, seq_count=3), N.KVQ_ERR_ARG), ({}, dict(seq_count=-1), N.KVQ_ERR_ARG),
    ({}, dict(count=-1), N.KVQ_ERR_ARG), ({}, dict(first=-1), N.KVQ_ERR_ARG), ({}, dict(out_dtype=2), N.KVQ_ERR_ARG),
    ({}, dict(cache=P + 128), N.KVQ_ERR_ALIGN), ({}, dict(k_out=P + 8), N.KVQ_ERR_ALIGN),
    ({}, dict(v_out=P + 8), N.KVQ_ERR_ALIGN), ({}, dict(starts=P + 2), N.KVQ_ERR_ALIGN),
    (dict(page_groups=2, num_pages=9), {}, N.KVQ_ERR_ARG)])
def test_read_refuses(kw, call, code):
    a = dict(cache=P, layer=0, seq_begin=0, seq_count=3, starts=None, first=0, count=4, k_out=P, v_out=P, out_dtype=0,
             stream=0)
    a.update(call)
    with pytest.raises(K.KvqError) as e:
        K.kvq_read_tokens(config(**kw), **a)
    assert e.value.code == code


def test_read_with_nothing_to_do():
    K.kvq_read_tokens(config(), P, 0, 0, 3, None, 0, 0, P, P, 0, 0)
    K.kvq_read_tokens(config(), P, 0, 0, 0, None, 0, 4, P, P, 0, 0)
    K.kvq_read_tokens(config(), P, 0, 0, 3, None, 0, 4, None, None, 0, 0)


@pytest.mark.parametrize("kw,call,code", [
    (dict(bits=3), {}, N.KVQ_ERR_ARG), ({}, dict(cache=None), N.KVQ_ERR_ARG), ({}, dict(q=None), N.KVQ_ERR_ARG),
    ({}, dict(k_draft=None), N.KVQ_ERR_ARG), ({}, dict(v_draft=None), N.KVQ_ERR_ARG), ({}, dict(out=None), N.KVQ_ERR_ARG),
    ({}, dict(workspace=None), N.KVQ_ERR_ARG), ({}, dict(layer=2), N.KVQ_ERR_ARG), ({}, dict(nodes=0), N.KVQ_ERR_ARG),
    ({}, dict(nodes=257), N.KVQ_ERR_ARG), ({}, dict(workspace_bytes=255), N.KVQ_ERR_WORKSPACE),
    ({}, dict(cache=P + 16), N.KVQ_ERR_ALIGN), ({}, dict(q=P + 2), N.KVQ_ERR_ALIGN),
    ({}, dict(k_draft=P + 2), N.KVQ_ERR_ALIGN), ({}, dict(v_draft=P + 2), N.KVQ_ERR_ALIGN),
    ({}, dict(out=P + 2), N.KVQ_ERR_ALIGN), ({}, dict(workspace=P + 16), N.KVQ_ERR_ALIGN),
    ({}, dict(n_nodes=P + 2), N.KVQ_ERR_ALIGN), (dict(scheme=1, in_dtype=1), {}, N.KVQ_ERR_UNSUPPORTED),
    (dict(q_heads=6), {}, N.KVQ_ERR_UNSUPPORTED), (dict(page_groups=2, num_pages=9), {}, N.KVQ_ERR_ARG)])
def test_tree_refuses(kw, call, code):
    a = dict(cache=P, layer=0, nodes=8, q=P, k_draft=P, v_draft=P, mask=None, n_nodes=None, softmax_scale=1.0, out=P,
             workspace=P, workspace_bytes=1 << 40, stream=0)
    a.update(call)
    with pytest.raises(K.KvqError) as e:
        K.kvq_tree_attention(config(**kw), **a)
    assert e.value.code == code


def test_tree_workspace():
    for kw in (dict(), dict(head_dim=256, bits=8, outliers=4, group_k=16, group_v=16), dict(scheme=4, head_dim=32)):
        sizes = [K.kvq_tree_workspace_bytes(config(**kw), n) for n in (1, 2, 16, 100, 256)]
        assert sizes == sorted(sizes) and sizes[0] >= 256
    for nodes in (0, -1, 257):
        with pytest.raises(K.KvqError):
            K.kvq_tree_workspace_bytes(config(), nodes)
    with pytest.raises(K.KvqError) as e:
        K.kvq_tree_workspace_bytes(config(scheme=2, in_dtype=1), 4)
    assert e.value.code == N.KVQ_ERR_UNSUPPORTED


def test_the_binding_refuses_tensors_that_the_library_would_misread():
    cache = K.QuantizedKVCache.__new__(K.QuantizedKVCache)
    cache.cfg, cache.device, cache._tree_workspaces = config(), torch.device("cuda", 0), {}
    q = torch.zeros(3, 4, 8, 128, dtype=torch.bfloat16)
    kv = torch.zeros(3, 4, 2, 128, dtype=torch.bfloat16)
    for bad in (dict(q=q.float()), dict(q=q[:2]), dict(q=q[0]), dict(k=kv[:, :2]), dict(v=kv.transpose(1, 2)),
                dict(mask=torch.zeros(3, 4, 4)), dict(mask=torch.zeros(3, 4, 3, dtype=torch.bool)),
                dict(n=torch.zeros(3)), {}):                       # {}: pageable host memory
        with pytest.raises(ValueError):
            cache.tree_decode(0, bad.get("q", q), bad.get("k", kv), bad.get("v", kv), mask=bad.get("mask"),
                              n_nodes=bad.get("n"))
    r = K.RotaryEmbedding(128)
    x = torch.zeros(5, 2, 128)
    for q_, k_, pos in ((None, None, None), (x, None, torch.zeros(5, dtype=torch.int32)), (x.double(), None, None),
                        (x, x, torch.zeros(4, dtype=torch.int32))):
        with pytest.raises(ValueError):
            r.rotate(q_, k_, pos)
    with pytest.raises(K.KvqError):
        K.RotaryEmbedding(128, rotary_dim=129)
