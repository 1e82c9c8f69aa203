"""What the packed operators and the many-tensor AdamW refuse, before any CUDA call:
sizes, null and unaligned pointers through the C entries, and the binding's own checks
of types, shapes and devices."""
import ctypes

import numpy as np
import pytest


@pytest.fixture(scope="module")
def L():
    import os
    from layer_streamed_qlora_nf4_b200 import build, lib
    if not os.path.exists(lib.LIB_PATH):
        build.build()
    lib.load()
    return lib


_raw = np.zeros(4096 + 64, np.uint8)
P = ctypes.c_void_p((_raw.ctypes.data + 63) // 64 * 64)    # aligned; never dereferenced
ODD = ctypes.c_void_p(P.value + 4)
HALF = ctypes.c_void_p(P.value + 16)


def _rc(L, name, *args):
    return getattr(L.load(), name)(*args)


def test_index_sizes(L):
    assert L.packed_index_ints(512, 5) == 8 + 4 * (9 + 9 + 7) + 3 * 512
    assert L.packed_index_ints(1, 1) == 8 + 4 * 3 + 3
    assert L.packed_index_ints(0, 1) == 0 and L.packed_index_ints(4, 0) == 0
    with pytest.raises(ValueError):
        L.PackedIndex(0, 1, device="cpu")


def test_packed_entries(L):
    bad = L.LSQ_ERR_INVALID, L.LSQ_ERR_SHAPE, L.LSQ_ERR_ALIGN, L.LSQ_ERR_WORKSPACE
    inval, shape, align, work = bad
    for rc, args in (
            (shape, (P, None, 1, 0, P, None)), (shape, (P, None, 0, 4, P, None)),
            (shape, (P, None, 1, (1 << 30) + 1, P, None)), (inval, (None, None, 1, 4, P, None)),
            (inval, (P, None, 1, 4, None, None)), (align, (P, None, 1, 4, ODD, None))):
        assert _rc(L, "packed_index", *args) == rc
    ok = [P, P, 1, 4, 4, 2, 64, P, P, None]
    for at, val, rc in ((0, None, inval), (1, None, inval), (2, 0, shape), (3, 0, shape),
                        (4, 3, shape), (4, 0, shape), (5, 0, shape), (6, 96, shape),
                        (7, None, inval), (8, None, inval), (0, ODD, align), (1, ODD, align),
                        (7, ODD, align), (7, HALF, align), (8, ODD, align), (3, 1 << 30, shape)):
        args = list(ok)
        args[at] = val
        if (at, val) == (3, 1 << 30):
            args[4] = 64
        assert _rc(L, "packed_attention_fwd", *args) == rc, (at, val)
    need = L.packed_attention_workspace_bytes(4, 4, 2, 64)
    assert need > 0
    for bad_shape in ((0, 4, 2, 64), (4, 3, 2, 64), (4, 4, 2, 32), (4, 0, 2, 64), (4, 4, 0, 64)):
        assert L.packed_attention_workspace_bytes(*bad_shape) == 0
    # sizes that the kernels' grids and counts have no room for
    for T, H, Hkv in ((1, 32768, 32768), (1 << 25, 32, 16)):
        assert L.packed_attention_workspace_bytes(T, H, Hkv, 64) == 0
        assert _rc(L, "packed_attention_fwd", P, P, 1, T, H, Hkv, 64, P, P, None) == shape
        assert _rc(L, "packed_attention_bwd", P, P, 1, P, P, P, T, H, Hkv, 64, P, P, 1 << 40,
                   None) == shape
    assert L.packed_attention_workspace_bytes((1 << 25) - 1, 32, 16, 64) > 0
    ok = [P, P, 1, P, P, P, 4, 4, 2, 64, P, P, need, None]
    for at, val, rc in ((0, None, inval), (3, None, inval), (4, None, inval), (5, None, inval),
                        (10, None, inval), (11, None, work), (12, need - 1, work),
                        (11, ODD, align), (11, HALF, align), (5, ODD, align),
                        (10, ODD, align), (10, HALF, align), (9, 80, shape),
                        (7, 5, shape)):
        args = list(ok)
        args[at] = val
        assert _rc(L, "packed_attention_bwd", *args) == rc, (at, val)
    ok = [P, P, 1, 4, None, P, P, 0, None]
    for at, val, rc in ((0, None, inval), (1, None, inval), (5, None, inval), (6, None, inval),
                        (7, 2, inval), (3, 0, shape)):
        args = list(ok)
        args[at] = val
        assert _rc(L, "packed_targets", *args) == rc, (at, val)
    ok = [P, 4, 9, P, None, None, P, P, P, 0, None]
    for at, val, rc in ((0, None, inval), (3, None, inval), (7, None, inval), (8, None, inval),
                        (1, 0, shape), (2, 0, shape), (9, 3, inval), (0, ODD, align),
                        (6, ODD, align), (1, 1 << 31, shape)):
        args = list(ok)
        args[at] = val
        assert _rc(L, "packed_cross_entropy", *args) == rc, (at, val)


def _table(L, *rows):
    t = (L.lsq_adamw_tensor * max(1, len(rows)))()
    for i, r in enumerate(rows):
        for k, v in dict(dict(p=P.value, g=P.value + 512, m=P.value + 1024, v=P.value + 1536,
                              m_scale=P.value + 2048, v_scale=P.value + 2112, n=16, lr=1e-3,
                              weight_decay=0.0), **r).items():
            setattr(t[i], k, v)
    return t


def _hyper(L, **kw):
    return L.lsq_adamw_hyper(**dict(dict(beta1=0.9, beta2=0.999, eps=1e-8, step=1, state_bits=8,
                                         grad_bits=32, step_dev=None), **kw))


def test_adamw_entries(L):
    inval, shape, align = L.LSQ_ERR_INVALID, L.LSQ_ERR_SHAPE, L.LSQ_ERR_ALIGN

    def rc(table, n, **kw):
        return _rc(L, "adamw_multi_step", table, n, ctypes.byref(_hyper(L, **kw)), None)
    for row, want in ((dict(p=None), inval), (dict(g=None), inval), (dict(m=None), inval),
                      (dict(v=None), inval), (dict(m_scale=None), inval), (dict(n=-1), shape),
                      (dict(p=P.value + 4), align), (dict(g=P.value + 8), align),
                      (dict(m=P.value + 1), align), (dict(v=P.value + 2), align),
                      (dict(v_scale=P.value + 2), align), (dict(lr=-1.0), inval),
                      (dict(lr=float("nan")), inval), (dict(weight_decay=float("inf")), inval)):
        assert rc(_table(L, row), 1) == want, row
    # the same tensor twice, one inside another, in and out of address order
    for a, b in ((0, 0), (0, 48), (48, 0)):
        assert rc(_table(L, dict(p=P.value + a), dict(p=P.value + b)), 2) == inval
    t = _table(L, {})
    for kw, want in ((dict(state_bits=16), inval), (dict(grad_bits=8), inval), (dict(step=0), shape),
                     (dict(beta1=1.0), inval), (dict(beta2=-0.1), inval), (dict(eps=0.0), inval),
                     (dict(eps=float("nan")), inval), (dict(beta1=float("nan")), inval)):
        assert rc(t, 1, **kw) == want, kw
    assert rc(t, -1) == shape
    assert _rc(L, "adamw_multi_step", t, 1, None, None) == inval
    assert _rc(L, "adamw_multi_step", None, 1, ctypes.byref(_hyper(L)), None) == inval
    assert [L.adamw_scale_floats(n) for n in (-1, 0, 1, 256, 257)] == [0, 0, 1, 1, 2]
    for name in ("adamw_state_dequantize", "adamw_state_quantize"):
        a = [P, P, 4, 1, P, None] if name.endswith("dequantize") else [P, 4, 1, P, P, None]
        sizes = (2, 3) if name.endswith("dequantize") else (1, 2)
        for at, val, want in ((0, None, inval), (sizes[0], 0, shape), (sizes[1], 2, inval),
                              (0, ODD, align)):
            args = list(a)
            args[at] = val
            assert _rc(L, name, *args) == want, (name, at, val)


def test_binding_checks(L):
    import torch
    i32 = torch.zeros(2, dtype=torch.int32)
    idx = L.PackedIndex(8, 2, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        L.packed_index(i32, idx)
    with pytest.raises(TypeError):
        L.packed_index(i32.long(), idx)
    with pytest.raises(ValueError):
        L.packed_index(torch.zeros(3, dtype=torch.int32), idx)
    with pytest.raises(ValueError):
        L.packed_index(i32, idx, prefix=torch.zeros(4, dtype=torch.int32)[::2][:1])
    qkv = torch.zeros(8, 8 * 64, dtype=torch.float16)
    o, lse = torch.zeros(8, 4 * 64, dtype=torch.float16), torch.zeros(4, 8)
    for a in ((qkv.float(), 4, 2, o, lse), (qkv, 4, 3, o, lse), (qkv, 0, 2, o, lse),
              (qkv[:4], 4, 2, o, lse), (qkv.t(), 4, 2, o, lse), (qkv, 4, 2, o[:, :64], lse),
              (qkv, 4, 2, o, lse.t()), (qkv, 4, 2, o.bfloat16(), lse)):
        with pytest.raises((TypeError, ValueError)):
            L.packed_attention_fwd(a[0], idx, *a[1:])
    with pytest.raises(ValueError, match="CUDA"):
        L.packed_attention_fwd(qkv, idx, 4, 2, o, lse)
    x = torch.zeros(3, 5)
    y, r, t = torch.zeros(3, dtype=torch.int32), torch.zeros(3), torch.zeros(1)
    for kw in (dict(dlogits=x), dict(weight=torch.zeros(2)), dict(count=t)):
        with pytest.raises((TypeError, ValueError)):
            L.packed_cross_entropy(x, y, r, t, **kw)
    with pytest.raises(ValueError):
        L.packed_cross_entropy(x[0], y, r, t)
    with pytest.raises(ValueError, match="CUDA"):
        L.packed_cross_entropy(x, y, r, t)
    p = [torch.zeros(300)]
    with pytest.raises(ValueError, match="CUDA"):
        L.AdamWMulti(p, p, p, p, lr=1.0)
    with pytest.raises(TypeError):
        L.AdamWMulti(p, [p[0].half()], p, p, lr=1.0)
    with pytest.raises(ValueError):
        L.AdamWMulti(p, p, p, [], lr=1.0)
    with pytest.raises(ValueError):
        L.AdamWMulti(p, p, p, p, lr=[1.0, 2.0])
    c = [torch.zeros(300, dtype=torch.int8)], [torch.zeros(300, dtype=torch.uint8)]
    with pytest.raises(ValueError):
        L.AdamWMulti(p, p, *c, lr=1.0, m_scale=[torch.zeros(1)], v_scale=[torch.zeros(2)])
    with pytest.raises(ValueError):
        L.AdamWMulti(p, p, *c, lr=1.0)
    with pytest.raises(TypeError):
        L.adamw_state_dequantize(p[0], p[0], p[0])
    assert L.AdamWMulti([], [], [], [], lr=1.0).step(1) is None


def _step_args(L, cfg):
    """Arguments of a packed step, right but for their device."""
    import torch
    n = L.lsq_lora_layout_get(cfg).floats_per_layer * cfg["n_layers"]
    V, D, T = cfg["vocab"], cfg["hidden"], 16
    return dict(tokens=torch.zeros(2, T, dtype=torch.int32),
                lengths=torch.zeros(2, 3, dtype=torch.int32),
                emb=torch.zeros(V, D, dtype=torch.bfloat16),
                lm_head=torch.zeros(V, D, dtype=torch.bfloat16),
                final_norm=torch.zeros(D, dtype=torch.bfloat16), lora=torch.zeros(n),
                lora_grad=torch.zeros(n), ws=torch.zeros(256, dtype=torch.uint8),
                logits_out=torch.zeros(T, V), prefix=torch.zeros(2, 3, dtype=torch.int32),
                loss_mask=torch.zeros(2, T, dtype=torch.bool))


def test_packed_step_binding(L):
    """Every tensor is checked for type, size and device before the library sees it."""
    from types import SimpleNamespace
    from layer_streamed_qlora_nf4_b200 import synth
    cfg = synth.SMALL
    stack = SimpleNamespace(cfg=L.cfg_struct(cfg), handle=None)
    ok = _step_args(L, cfg)
    with pytest.raises(ValueError, match="CUDA"):
        L.stream_stack_packed_step(stack, **ok)
    for name in ok:
        t = ok[name]
        wrong = [t.double(), t.reshape(-1)[:-1], [0]]
        if t.dim() == 2:
            wrong += [t[:, :-1], t.t().contiguous().t()]
        for w in wrong:
            if name == "ws" and w is wrong[1]:
                continue                 # (its length is the library's to judge)
            with pytest.raises((TypeError, ValueError, AttributeError)) as e:
                L.stream_stack_packed_step(stack, **dict(ok, **{name: w}))
            assert "CUDA" not in str(e.value), (name, str(e.value))


def test_packed_layer_binding(L):
    import torch
    from layer_streamed_qlora_nf4_b200 import synth
    cfg, T = synth.SMALL, 8
    idx = L.PackedIndex(T, 2, device="cpu")
    x = torch.zeros(T, cfg["hidden"])
    n = L.lsq_lora_layout_get(cfg).floats_per_layer
    blob = torch.zeros(L.lsq_layer_layout_get(cfg).bytes, dtype=torch.uint8)
    lora, ws = torch.zeros(n), torch.zeros(256, dtype=torch.uint8)
    for b, l, w in ((blob[:-1], lora, ws), (blob.int(), lora, ws), (blob, lora[:-1], ws),
                    (blob, lora.half(), ws), (blob, lora, ws.float()), (blob, lora, None),
                    (None, lora, ws)):
        with pytest.raises((TypeError, ValueError)) as e:
            L.decoder_layer_packed_fwd(cfg, b, l, x, idx, x, w)
        assert "CUDA" not in str(e.value)
        with pytest.raises((TypeError, ValueError)) as e:
            L.decoder_layer_packed_bwd(cfg, b, l, x, x, idx, x, lora, w)
        assert "CUDA" not in str(e.value)
    for l, g in ((None, lora), (lora, None), (lora, lora[1:])):
        with pytest.raises((TypeError, ValueError)) as e:
            L.decoder_layer_packed_bwd(cfg, blob, l, x, x, idx, x, g, ws)
        assert "CUDA" not in str(e.value)
    for l in (lora, None):               # (no adapter: the forward takes it)
        with pytest.raises(ValueError, match="CUDA"):
            L.decoder_layer_packed_fwd(cfg, blob, l, x, idx, x, ws)


def test_a_step_count_on_the_host_is_refused(L):
    """A count that the device is to read must lie on it."""
    import torch
    from types import SimpleNamespace
    from layer_streamed_qlora_nf4_b200 import synth
    opt = L.AdamWMulti([], [], [], [], lr=1.0)
    seen = []
    keep = L._call
    L._call = lambda name, stream, tensors, *a, **k: seen.append(tensors)
    try:
        count = torch.ones(1, dtype=torch.int32)
        L.stream_stack_packed_step(SimpleNamespace(cfg=L.cfg_struct(synth.SMALL), handle=None),
                                   opt=opt, step=count, **_step_args(L, synth.SMALL))
    finally:
        L._call = keep
    assert any(t is count for t in seen[0])


def test_rates_need_one_number_per_tensor(L):
    o = L.AdamWMulti([], [], [], [], lr=1.0)
    o.set_rates(0.5)
    o.set_rates([], weight_decay=[])
    for bad in (dict(lr=[1.0]), dict(lr=1.0, weight_decay=[1.0])):
        with pytest.raises(ValueError):
            o.set_rates(**bad)
        with pytest.raises(ValueError):
            L.AdamWMulti([], [], [], [], **bad)


def test_a_new_index_holds_no_documents(L):
    """What the operators take their rows from is never unwritten memory."""
    import torch
    junk = [torch.full((L.packed_index_ints(5000, 7),), -1, dtype=torch.int32) for _ in range(4)]
    del junk                                       # (memory that the next buffers may reuse)
    for _ in range(4):
        assert not L.PackedIndex(5000, 7, device="cpu").buf.any()
