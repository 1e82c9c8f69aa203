"""The packed operators and AdamW where element offsets pass 2^31, and two calls at once: what a
document, a row or a block gets does not depend on where it lies or on what else runs, so each is
compared bit for bit with a small call of its own."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from layer_streamed_qlora_nf4_b200 import lib
    lib.load()
    return lib


@pytest.fixture(autouse=True)
def _give_back():
    """The tens of GB of a test go back to the device."""
    yield
    import torch
    torch.cuda.empty_cache()


def _attention(L, qkv, dout, lengths, prompts, H, Hkv, stream=None):
    import torch
    T, d = qkv.shape[0], qkv.shape[1] // (H + 2 * Hkv)
    idx = L.PackedIndex(T, len(lengths))
    L.packed_index(torch.tensor(lengths, dtype=torch.int32, device="cuda"), idx,
                   prefix=torch.tensor(prompts, dtype=torch.int32, device="cuda"))
    o = torch.empty(T, H * d, dtype=torch.float16, device="cuda")
    lse, dqkv = torch.empty(H, T, device="cuda"), torch.empty(qkv.shape, dtype=torch.bfloat16,
                                                              device="cuda")
    ws = torch.empty(L.packed_attention_workspace_bytes(T, H, Hkv, d), dtype=torch.uint8,
                     device="cuda")
    L.packed_attention_fwd(qkv, idx, H, Hkv, o, lse)
    L.packed_attention_bwd(qkv, idx, o, lse, dout, H, Hkv, dqkv, ws)
    return o, lse, dqkv


def test_attention_behind_2_31_elements(L):
    import torch
    H, Hkv, d = 32, 8, 128
    rng = np.random.default_rng(0)
    lengths = rng.integers(200, 900, 660).tolist()
    prompts = [int(rng.integers(0, n + 1)) if i % 2 else 0 for i, n in enumerate(lengths)]
    T = sum(lengths) + 50
    assert T * (H + 2 * Hkv) * d > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.empty(T, (H + 2 * Hkv) * d, dtype=torch.float16, device="cuda").normal_(generator=g)
    dout = torch.empty(T, H * d, dtype=torch.bfloat16, device="cuda").normal_(generator=g).mul_(1e-5)
    o, lse, dqkv = _attention(L, qkv, dout, lengths, prompts, H, Hkv)
    last = slice(T - 50 - sum(lengths[-40:]), T)           # the last 40 documents and the padding
    so, slse, sdqkv = _attention(L, qkv[last].clone(), dout[last].clone(), lengths[-40:],
                                 prompts[-40:], H, Hkv)
    assert torch.equal(o[last], so) and torch.equal(lse[:, last], slse)
    assert torch.equal(dqkv[last], sdqkv) and sdqkv[:-50].float().abs().sum(1).min() > 0
    assert not o[-50:].any() and not dqkv[-50:].any()
    assert L.lsq_device_status(clear=True) == 0


def test_loss_behind_2_31_logits(L):
    import torch
    T, V = 16500, 131075                                   # (rows that begin at odd elements)
    assert T * V > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty(T, V, device="cuda").normal_(generator=g)
    y = torch.randint(-1, V, (T,), device="cuda", generator=g, dtype=torch.int32)
    y[:-300:3] = -1

    def run(x, y):
        n = x.shape[0]
        rl, tot = torch.empty(n, device="cuda"), torch.empty(1, device="cuda")
        dl = torch.empty(n, V, dtype=torch.bfloat16, device="cuda")
        L.packed_cross_entropy(x, y, rl, tot, dlogits=dl)
        return rl, dl
    rl, dl = run(x, y)
    k = T - 300                                            # (a multiple of 8 rows from the start)
    assert k * V % 8 == 0
    srl, sdl = run(x[k:].clone(), y[k:].clone())
    assert torch.equal(rl[k:], srl) and torch.equal(dl[k:], sdl)
    assert L.lsq_device_status(clear=True) == 0


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_behind_2_31_elements(L, bits):
    import torch
    n, tail = 2 ** 31 + 256 * 5 + 77, 256 * 9 + 77
    g = torch.Generator(device="cuda").manual_seed(3)

    def tensors(n):
        mdt, vdt = (torch.int8, torch.uint8) if bits == 8 else (torch.float32, torch.float32)
        k = L.adamw_scale_floats(n)
        return (torch.zeros(n, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(n, dtype=mdt, device="cuda"), torch.zeros(n, dtype=vdt, device="cuda"),
                torch.zeros(k, device="cuda"), torch.zeros(k, device="cuda"))
    big, small = tensors(n), tensors(tail)
    small[0].normal_(generator=g)
    small[1].normal_(generator=g).mul_(1e-4)
    for b, s in zip(big[:2], small[:2]):
        b[n - tail:] = s
    for p, gr, m, v, ms, vs in (big, small):
        o = L.AdamWMulti([p], [gr], [m], [v], lr=1e-3, weight_decay=0.01,
                         m_scale=[ms] if bits == 8 else None, v_scale=[vs] if bits == 8 else None)
        o.step(1)
        o.step(2)
    for b, s in zip(big, small):
        assert torch.equal(b[len(b) - len(s):], s)
    assert not big[0][:n - tail].any() and not big[2][:n - tail].any() and small[2].any()
    if bits == 8:
        out, ref = torch.empty(n, device="cuda"), torch.empty(tail, device="cuda")
        L.adamw_state_dequantize(big[3], big[5], out)
        L.adamw_state_dequantize(small[3], small[5], ref)
        assert torch.equal(out[n - tail:], ref) and ref.any()
    assert L.lsq_device_status(clear=True) == 0


def test_two_calls_at_once(L):
    """Two streams with their own rows, indexes, outputs and workspaces; a third with a loss and
    an update."""
    import torch
    rng = np.random.default_rng(5)
    jobs = []
    for H, Hkv, d, n in ((16, 2, 128, 9), (8, 2, 64, 30)):
        lengths = rng.integers(1, 400, n).tolist()
        T = sum(lengths) + 3
        g = torch.Generator(device="cuda").manual_seed(n)
        qkv = torch.empty(T, (H + 2 * Hkv) * d, dtype=torch.float16, device="cuda").normal_(generator=g)
        dout = torch.empty(T, H * d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        jobs.append((qkv, dout, lengths, [k // 3 for k in lengths], H, Hkv))
    x, y = torch.randn(300, 5003, device="cuda"), torch.randint(0, 5003, (300,), device="cuda").int()

    def loss():
        rl, tot = torch.empty(300, device="cuda"), torch.empty(1, device="cuda")
        dl = torch.empty(300, 5003, dtype=torch.bfloat16, device="cuda")
        L.packed_cross_entropy(x, y, rl, tot, dlogits=dl)
        p, gr = dl.float().view(-1)[:100000].contiguous(), dl.view(-1)[:100000].contiguous()
        m, v = torch.zeros_like(p), torch.zeros_like(p)
        L.AdamWMulti([p], [gr], [m], [v], lr=1e-3).step(1)
        return rl, tot, dl, p, m, v
    want = [_attention(L, *j) for j in jobs] + [loss()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(10):
        got = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append(_attention(L, *jobs[i]) if i < 2 else loss())
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert L.lsq_device_status(clear=True) == 0
