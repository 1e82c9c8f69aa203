"""GPU parity of AdamW over many tensors: the 8-bit codes and scales bit for bit, the
fp32 moments bit for bit, and the parameters within a few fp32 roundings of the oracle.
"""
import numpy as np
import pytest

from oracle import packed as op

pytestmark = pytest.mark.gpu

SIZES = [1, 3, 4, 255, 256, 257, 0, 2048, 2049, 5000, 64 * 256]


@pytest.fixture(scope="module")
def L():
    from layer_streamed_qlora_nf4_b200 import lib
    lib.load()
    return lib


def _problem(sizes, bits, gbf16, seed):
    """Tensors with a running state, every one in its own allocation."""
    import torch
    rng = np.random.default_rng(seed)
    out = dict(p=[], g=[], m=[], v=[], ms=[], vs=[])
    for n in sizes:
        s = np.exp(rng.standard_normal()) * 1e-4
        g = (rng.standard_normal(n) * s).astype(np.float32)
        if gbf16:
            g = torch.from_numpy(g).bfloat16().float().numpy()
        m = (rng.standard_normal(n) * s * 0.3).astype(np.float32)
        v = ((0.1 + rng.standard_normal(n) ** 2) * s * s).astype(np.float32)
        v[rng.random(n) < 0.05] = 0
        if bits == 8:
            mc, ms = op.encode(m, True)
            vc, vs = op.encode(v, False)
            out["m"].append(mc), out["v"].append(vc), out["ms"].append(ms), out["vs"].append(vs)
        else:
            out["m"].append(m), out["v"].append(v), out["ms"].append(None), out["vs"].append(None)
        out["p"].append((rng.standard_normal(n) * 0.02 * (rng.random() < 0.7)).astype(np.float32))
        out["g"].append(g)
    return out


def _device(x, gbf16):
    import torch
    d = {k: [None if a is None else torch.from_numpy(a.copy()).cuda() for a in x[k]] for k in x}
    if gbf16:
        d["g"] = [a.bfloat16() for a in d["g"]]
    return d


def _opt(L, d, lr, wd, bits):
    return L.AdamWMulti(d["p"], d["g"], d["m"], d["v"], lr=lr, weight_decay=wd,
                        m_scale=d["ms"] if bits == 8 else None,
                        v_scale=d["vs"] if bits == 8 else None)


def _reference(x, step, lr, wd, bits):
    """One oracle step of every tensor, in place."""
    for i in range(len(x["p"])):
        m, v = x["m"][i], x["v"][i]
        if bits == 8:
            m, v = op.decode(m, x["ms"][i]), op.decode(v, x["vs"][i])
        p, m, v = op.adamw(x["p"][i], x["g"][i], m, v, step, lr[i], wd[i])
        x["p"][i] = p
        if bits == 8:
            x["m"][i], x["ms"][i] = op.encode(m, True)
            x["v"][i], x["vs"][i] = op.encode(v, False)
        else:
            x["m"][i], x["v"][i] = m, v


def _check(x, d, lr, bits, steps=1):
    for i in range(len(x["p"])):
        for k in ("m", "v") + (("ms", "vs") if bits == 8 else ()):
            assert np.array_equal(d[k][i].cpu().numpy(), x[k][i]), (k, i)
        # p is rounded once a step (2^-24), and the update of at most a few lr is off by
        # 2^-20 relative
        tol = steps * (2.0 ** -23 * np.abs(x["p"][i]) + 2.0 ** -20 * 10 * lr[i])
        assert (np.abs(d["p"][i].cpu().numpy() - x["p"][i]) <= tol).all(), i


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("gbf16", [False, True])
@pytest.mark.parametrize("copies", [1, 50])
def test_steps(L, bits, gbf16, copies):
    """copies = 50: more tensors than one launch takes."""
    import torch
    sizes = SIZES * copies if copies == 1 else [s for s in SIZES if s < 300] * copies + [700]
    sizes = sizes if copies == 1 else sizes * 2
    x = _problem(sizes, bits, gbf16, seed=bits + copies)
    d = _device(x, gbf16)
    n = len(sizes)
    lr = [2e-4 * (1 + i % 3) for i in range(n)]
    wd = [0.01 * (i % 2) for i in range(n)]
    o = _opt(L, d, lr, wd, bits)
    for step in (3, 4):
        o.step(step)
        _reference(x, step, lr, wd, bits)
    torch.cuda.synchronize()
    assert L.lsq_device_status(clear=True) == 0
    _check(x, d, lr, bits, steps=2)


@pytest.mark.parametrize("bits", [8, 32])
def test_from_nothing(L, bits):
    """Zero state and zero parameters: the first step is lr times the gradient's sign."""
    import torch
    n = 1000
    g = np.random.default_rng(0).standard_normal(n).astype(np.float32) * np.float32(1e-6)
    g[::7] = 0
    x = dict(p=[np.zeros(n, np.float32)], g=[g],
             m=[np.zeros(n, np.int8 if bits == 8 else np.float32)],
             v=[np.zeros(n, np.uint8 if bits == 8 else np.float32)],
             ms=[np.zeros(4, np.float32)], vs=[np.zeros(4, np.float32)])
    d = _device(x, False)
    _opt(L, d, 1e-3, 0.0, bits).step(1)
    _reference(x, 1, [1e-3], [0.0], bits)
    torch.cuda.synchronize()
    _check(x, d, [1e-3], bits)
    assert not d["p"][0][::7].any()


def test_tiny_and_huge_moments(L):
    """Blocks whose largest magnitude is below the normal range are stored as zeros; very
    large ones stay finite."""
    import torch
    g = np.concatenate([np.full(256, 1e-39), np.full(256, 1e-22), np.full(256, 1e15)]).astype(np.float32)
    x = dict(p=[np.zeros(768, np.float32)], g=[g], m=[np.zeros(768, np.int8)],
             v=[np.zeros(768, np.uint8)], ms=[np.zeros(3, np.float32)], vs=[np.zeros(3, np.float32)])
    d = _device(x, False)
    _opt(L, d, 1e-3, 0.0, 8).step(1)
    _reference(x, 1, [1e-3], [0.0], 8)
    torch.cuda.synchronize()
    _check(x, d, [1e-3], 8)
    assert d["ms"][0][0].item() == 0 and d["vs"][0][1].item() == 0


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("eps", [1e-30, 2.0 ** -126])
def test_denominators_of_subnormal_and_huge_moments(L, bits, eps):
    """With an eps far below the root of a subnormal v that root is the denominator.  The
    change of p (from 0) is a product of rate, moment and reciprocal: the rate is rounded
    twice, the root and the reciprocal are off by 2^-23, the root's factor, the sum, and
    three products by 2^-24 each, together below 2^-20; its last bits may be subnormal."""
    import torch
    n = 2048
    rng = np.random.default_rng(5)
    g = (rng.standard_normal(n) * 10.0 ** rng.uniform(-21.5, -16.5, n)).astype(np.float32)
    g[512:1024:3] = 10.0 ** rng.uniform(14, 17, len(g[512:1024:3]))
    x = dict(p=[np.zeros(n, np.float32)], g=[g],
             m=[np.zeros(n, np.int8 if bits == 8 else np.float32)],
             v=[np.zeros(n, np.uint8 if bits == 8 else np.float32)],
             ms=[np.zeros(8, np.float32)], vs=[np.zeros(8, np.float32)])
    d = _device(x, False)
    L.AdamWMulti(d["p"], d["g"], d["m"], d["v"], lr=1e-3, m_scale=d["ms"] if bits == 8 else None,
                 v_scale=d["vs"] if bits == 8 else None, eps=eps).step(1)
    torch.cuda.synchronize()
    assert L.lsq_device_status(clear=True) == 0
    zero = np.zeros(n, np.float32)
    rp, m1, v1 = op.adamw(zero, g, zero, zero, 1, 1e-3, 0.0, eps=eps)
    assert ((v1 > 0) & (v1 < 2.0 ** -126)).sum() > 100 and (v1 > 2.0 ** 100).sum() > 10
    got = d["p"][0].cpu().numpy().astype(np.float64)
    ok = np.abs(rp) < 3e38
    assert (np.abs(got - rp)[ok] <= 2.0 ** -20 * np.abs(rp[ok]) + 2.0 ** -149).all()
    for k, s, ref, signed in (("m", "ms", m1, True), ("v", "vs", v1, False)):
        if bits == 8:
            c, sc = op.encode(ref, signed)
            assert np.array_equal(d[k][0].cpu().numpy(), c)
            assert np.array_equal(d[s][0].cpu().numpy(), sc)
        else:
            assert np.array_equal(d[k][0].cpu().numpy(), ref)


@pytest.mark.parametrize("bits", [8, 32])
def test_not_finite_gradients_are_left_out(L, bits):
    import torch
    sizes = [600]
    x = _problem(sizes, bits, False, 7)
    bad = [0, 5, 256, 599]
    clean = {k: [a.copy() if a is not None else None for a in v] for k, v in x.items()}
    for i, val in zip(bad, (np.nan, np.inf, -np.inf, 1e30)):  # 1e30: its square overflows
        x["g"][0][i] = val
    d = _device(x, False)
    _opt(L, d, 1e-3, 0.01, bits).step(2)
    torch.cuda.synchronize()
    assert L.lsq_device_status(clear=True) == L.LSQ_DEV_ERR_NONFINITE
    p = d["p"][0].cpu().numpy()
    assert np.array_equal(p[bad], clean["p"][0][bad]) and np.isfinite(p).all()
    m0 = clean["m"][0] if bits == 32 else op.decode(clean["m"][0], clean["ms"][0])
    v0 = clean["v"][0] if bits == 32 else op.decode(clean["v"][0], clean["vs"][0])
    g = clean["g"][0].copy()
    rp, m1, v1 = op.adamw(clean["p"][0], g, m0, v0, 2, 1e-3, 0.01)
    m1[bad], v1[bad], rp[bad] = m0[bad], v0[bad], clean["p"][0][bad]
    if bits == 32:
        assert np.array_equal(d["m"][0].cpu().numpy(), m1)
        assert np.array_equal(d["v"][0].cpu().numpy(), v1)
    else:
        for k, s, ref, signed in (("m", "ms", m1, True), ("v", "vs", v1, False)):
            c, sc = op.encode(ref, signed)
            assert np.array_equal(d[k][0].cpu().numpy(), c)
            assert np.array_equal(d[s][0].cpu().numpy(), sc)


@pytest.mark.parametrize("which", ["ms", "vs"])
@pytest.mark.parametrize("value", [np.nan, np.inf])
@pytest.mark.parametrize("n", [1, 3, 44, 255, 256])
def test_a_scale_that_is_not_finite_in_a_short_last_block(L, n, value, which):
    """A damaged 8-bit state.  Elements whose moments are not finite keep their parameter, and
    such a moment is zero afterwards; the elements before the block are updated as ever, and
    nothing behind the tensor is touched."""
    import torch
    x = _problem([256 + n], 8, False, 3)
    x["m"][0][256::2] = 0            # codes 0 and others: 0 * inf and c * inf
    x["v"][0][256::3] = 0
    x[which][0][1] = value
    d = _device(x, False)
    # the tensor's arrays lie in front of values that must stay
    d["p"][0] = torch.cat([d["p"][0], torch.full((300,), 7.5, device="cuda")])
    d["m"][0] = torch.cat([d["m"][0], torch.full((300,), 77, dtype=torch.int8, device="cuda")])
    d["v"][0] = torch.cat([d["v"][0], torch.full((300,), 77, dtype=torch.uint8, device="cuda")])
    behind = {k: d[k][0][256 + n:].clone() for k in ("p", "m", "v")}
    view = {k: [d[k][0][:256 + n]] for k in ("p", "m", "v")}
    _opt(L, dict(d, **view), 1e-3, 0.01, 8).step(2)
    torch.cuda.synchronize()
    assert L.lsq_device_status(clear=True) == L.LSQ_DEV_ERR_NONFINITE
    p = view["p"][0].cpu().numpy()
    assert np.array_equal(p[256:], x["p"][0][256:])
    for k in ("p", "m", "v"):
        assert torch.equal(d[k][0][256 + n:], behind[k])
    assert np.isfinite(d["ms"][0].cpu().numpy()).all() and np.isfinite(d["vs"][0].cpu().numpy()).all()
    bad = dict(ms="m", vs="v")[which]
    assert d[which][0][1].item() == 0 and not view[bad][0][256:].any()
    first = {k: [x[k][0][:1 if k in ("ms", "vs") else 256]] for k in x}
    p0 = first["p"][0].astype(np.float64)
    _reference(first, 2, [1e-3], [0.01], 8)
    for k in ("m", "v", "ms", "vs"):
        got = view[k][0][:256] if k in view else d[k][0][:1]
        assert np.array_equal(got.cpu().numpy(), first[k][0]), k
    # p is rounded once (2^-24); its change, the decay lr wd p and the rest, has the roundings
    # counted in test_denominators_of_subnormal_and_huge_moments, together below 2^-20.  (With v
    # of 0 and a small gradient the change is some hundred lr, so it is taken as it is.)
    decay = 1e-3 * 0.01 * np.abs(p0)
    tol = 2.0 ** -23 * np.abs(first["p"][0]) + 2.0 ** -20 * (np.abs(first["p"][0] - p0) + 2 * decay)
    worst = (np.abs(p[:256] - first["p"][0]) / np.maximum(tol, 1e-45)).max()
    assert worst <= 1, worst


def test_replayed_graph_follows_the_count(L):
    import torch
    x = _problem([700, 300], 8, False, 9)
    d = _device(x, False)
    count = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = _opt(L, d, 1e-3, 0.0, 8)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        count += 1
        o.step(count)
    for step in (1, 2, 3):
        g.replay()
        _reference(x, step, [1e-3] * 2, [0.0] * 2, 8)
    torch.cuda.synchronize()
    _check(x, d, [1e-3] * 2, 8, steps=3)


@pytest.mark.parametrize("n", [1, 15, 16, 257, 4096, 70001])
@pytest.mark.parametrize("signed", [True, False])
def test_state_round_trip(L, n, signed):
    import torch
    rng = np.random.default_rng(n)
    v = (rng.standard_normal(n) * np.exp(3 * rng.standard_normal(n))).astype(np.float32)
    v = v if signed else np.abs(v)
    codes, scale = op.encode(v, signed)
    c = torch.full((n,), 3, dtype=torch.int8 if signed else torch.uint8, device="cuda")
    s = torch.full((len(scale),), 9.0, device="cuda")
    L.adamw_state_quantize(torch.from_numpy(v).cuda(), c, s)
    assert np.array_equal(c.cpu().numpy(), codes) and np.array_equal(s.cpu().numpy(), scale)
    out = torch.empty(n, device="cuda")
    L.adamw_state_dequantize(c, s, out)
    assert np.array_equal(out.cpu().numpy(), op.decode(codes, scale))


def test_every_code_and_its_borders(L):
    """Values at, one step below and one step above every border between two codes."""
    import torch
    for signed, top, pw in ((True, 127, 2), (False, 255, 4)):
        edge = (((2 * np.arange(top) + 1) / (2.0 * top)) ** pw).astype(np.float32)
        vals = np.concatenate([edge, np.nextafter(edge, np.float32(0)),
                               np.nextafter(edge, np.float32(2))])
        for a in (1.0, 3e-7, 12345.678):
            x = (vals * np.float32(a)).astype(np.float32)
            x = np.resize(x, (len(x) + 254) // 255 * 255).reshape(-1, 255)
            x = np.concatenate([np.full((len(x), 1), a, np.float32), x], 1).reshape(-1)
            codes, scale = op.encode(x, signed)
            c = torch.empty(len(x), dtype=torch.int8 if signed else torch.uint8, device="cuda")
            s = torch.empty(len(scale), device="cuda")
            L.adamw_state_quantize(torch.from_numpy(x).cuda(), c, s)
            assert np.array_equal(c.cpu().numpy(), codes)


def test_borders_closer_than_fp64_products_tell(L):
    """x 510^4 and a (2 b + 1)^4 have up to 60 bits: where their fp64 products are equal, the
    code is still that of the exact comparison.  In the update, and in the conversion."""
    import torch
    pairs = np.array([[10322846, 665658.125], [8629209, 3499999], [15995371, 7.3828125],
                      [16777215, 16646655]], np.float32)
    # 665658.125 510^4 - 10322846 257^4 = 4, 3499999 510^4 - 8629209 407^4 = -72
    want = [129, 203]
    x = np.zeros((len(pairs), 256), np.float32)
    x[:, 0], x[:, 1:3] = pairs[:, 0], pairs[:, 1:]
    # a few fp32 steps to both sides of every border, for scales of 24 bits
    rng = np.random.default_rng(0)
    a = (rng.integers(1 << 23, 1 << 24, 300) * 2.0 ** rng.integers(-60, 60, 300)).astype(np.float32)
    near = a[:, None].astype(np.float64) * ((2 * np.arange(255) + 1) / 510.0) ** 4
    for step in (-1, 0, 1):
        e = near.astype(np.float32)
        e = e if step == 0 else np.nextafter(e, np.float32(0 if step < 0 else np.inf))
        x = np.concatenate([x, np.concatenate([a[:, None], e], 1)])
    x = x.reshape(-1)
    codes, scale = op.encode(x, False)
    assert [codes[256 * i + 1] for i in (0, 1)] == want
    c = torch.empty(len(x), dtype=torch.uint8, device="cuda")
    s = torch.empty(len(scale), device="cuda")
    L.adamw_state_quantize(torch.from_numpy(x).cuda(), c, s)
    assert np.array_equal(c.cpu().numpy(), codes) and np.array_equal(s.cpu().numpy(), scale)
    # the update: v = (g - 0 g) g with beta2 = 0 and a zero state is g^2, rounded once
    g = np.sqrt(x.astype(np.float64)).astype(np.float32)
    d = dict(p=[torch.zeros(len(x), device="cuda")], g=[torch.from_numpy(g).cuda()],
             m=[torch.zeros(len(x), dtype=torch.int8, device="cuda")], v=[c.zero_()],
             ms=[torch.zeros(len(scale), device="cuda")], vs=[s.zero_()])
    L.AdamWMulti(d["p"], d["g"], d["m"], d["v"], lr=0.0, m_scale=d["ms"], v_scale=d["vs"],
                 betas=(0.0, 0.0)).step(1)
    codes, scale = op.encode(g * g, False)
    assert np.array_equal(c.cpu().numpy(), codes) and np.array_equal(s.cpu().numpy(), scale)
    assert L.lsq_device_status(clear=True) == 0


@pytest.mark.parametrize("bits", [8, 32])
def test_rates_follow_a_schedule(L, bits):
    """Warm-up and decay, by one number and by one per tensor; a bad rate is refused at the step
    and changes nothing."""
    import torch
    x = _problem([700, 300, 1], bits, False, 21)
    d = _device(x, False)
    o = _opt(L, d, 1e-3, 0.01, bits)
    wd = [0.01] * 3
    for step, lr in ((1, 0.0), (2, [1e-4, 2e-4, 0.0]), (3, 1e-3), (4, [5e-4, 1e-4, 2e-4])):
        if step == 3:
            wd = [0.0, 0.1, 0.02]
        o.set_rates(lr, weight_decay=wd if step == 3 else None)
        o.step(step)
        lrs = lr if isinstance(lr, list) else [lr] * 3
        before = [p.copy() for p in x["p"]]
        _reference(x, step, lrs, wd, bits)
        # the parameters are compared step by step, each from the device's own
        for i in range(3):
            got = d["p"][i].cpu().numpy()
            decay = lrs[i] * wd[i] * np.abs(before[i].astype(np.float64))
            tol = (2.0 ** -23 * np.abs(x["p"][i]) +
                   2.0 ** -20 * (np.abs(x["p"][i] - before[i]) + 2 * decay))
            assert (np.abs(got - x["p"][i]) <= tol).all(), (step, i)
            x["p"][i] = got
            for k in ("m", "v") + (("ms", "vs") if bits == 8 else ()):
                assert np.array_equal(d[k][i].cpu().numpy(), x[k][i]), (k, i)
    kept = [t.clone() for k in ("p", "m", "v") for t in d[k]]
    for bad in (-1.0, float("nan"), float("inf")):
        o.set_rates([1e-3, bad, 1e-3])
        with pytest.raises(L.LsqError) as e:
            o.step(5)
        assert e.value.code == L.LSQ_ERR_INVALID
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, [t for k in ("p", "m", "v") for t in d[k]]))
    assert L.lsq_device_status(clear=True) == 0
