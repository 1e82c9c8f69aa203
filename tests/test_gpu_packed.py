"""GPU parity of the packed operators (index, targets, attention inside documents,
cross-entropy) against the fp64 oracle.

Tolerances count roundings.  A rounding is off by at most half a step: 2^-11 relative
in fp16, 2^-9 in bf16 (8 significant bits, so half a step is 2^-9 of the power of two
above and 2^-8 of the value at worst: 2^-8 is used), 2^-24 in fp32.
Scores: |q||k| sums in fp32 by the tensor cores (each of d products, steps of 2^-23),
times log2 e: below 2^-15 for the values here, so p = exp2(s - m) is off by at most
2^-15 relative from fp32 work.
"""
import numpy as np
import pytest

from oracle import packed as op

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -15     # fp32 work on scores and sums, as above
HALF = 2.0 ** -11    # half a step of fp16
BF = 2.0 ** -8       # half a step of bf16

HEADS = [(8, 2, 64), (4, 4, 128), (6, 2, 128), (5, 1, 64), (4, 1, 128)]
ROWS = [
    # lengths, prompts, tokens
    ([1], None, 1),
    ([1], None, 3),
    ([128], None, 128),
    ([129], [129], 129),
    ([127, 1, 0, 129, 200], None, 500),
    ([64, 64, 0, 0, 65, 63], [64, 1, 0, 0, 0, 30], 256),
    ([3] * 41, [2] * 41, 140),
    ([700], None, 701),
    ([300, 280], [140, 200], 600),
    ([0, 0, 5], None, 9),
    ([0], None, 4),
]


@pytest.fixture(scope="module")
def L():
    from layer_streamed_qlora_nf4_b200 import lib
    lib.load()
    return lib


def _index(L, lengths, prefix, T):
    import torch
    idx = L.PackedIndex(T, len(lengths))
    idx.buf.fill_(-7)
    L.packed_index(torch.tensor(lengths, dtype=torch.int32, device="cuda"), idx,
                   prefix=None if prefix is None else torch.tensor(prefix, dtype=torch.int32,
                                                                   device="cuda"))
    return idx


def _inputs(T, H, Hkv, d, seed, grad=1e-5):
    import torch
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, (H + 2 * Hkv) * d, generator=g).half()
    dout = (torch.randn(T, H * d, generator=g) * torch.exp(torch.randn(T, 1, generator=g)) *
            grad).bfloat16()
    return qkv, dout


def _run(L, qkv, dout, idx, H, Hkv, ws_fill=255):
    import torch
    T, d = qkv.shape[0], qkv.shape[1] // (H + 2 * Hkv)
    nan = float("nan")
    o = torch.full((T, H * d), nan, dtype=torch.float16, device="cuda")
    lse = torch.full((H, T), nan, device="cuda")
    dqkv = torch.full((T, (H + 2 * Hkv) * d), nan, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((L.packed_attention_workspace_bytes(T, H, Hkv, d),), ws_fill, dtype=torch.uint8,
                    device="cuda")
    L.packed_attention_fwd(qkv, idx, H, Hkv, o, lse)
    L.packed_attention_bwd(qkv, idx, o, lse, dout, H, Hkv, dqkv, ws)
    torch.cuda.synchronize()
    assert L.lsq_device_status(clear=True) == 0
    return o, lse, dqkv


def _check(qkv, dout, docs, H, Hkv, o, lse, dqkv):
    x = qkv.float().numpy().astype(np.float64)
    T, d = x.shape[0], x.shape[1] // (H + 2 * Hkv)
    q, k, v = op.split_heads(x, H, Hkv)
    ro, rlse, p = op.attention_fwd(x, H, Hkv, docs)
    rg = op.attention_bwd(x, H, Hkv, docs, dout.float().numpy())
    do = dout.float().numpy().astype(np.float64).reshape(T, H, d)
    o = o.float().cpu().numpy().astype(np.float64).reshape(T, H, d)
    lse = lse.cpu().numpy()
    got = dqkv.float().cpu().numpy().astype(np.float64).reshape(T, H + 2 * Hkv, d)
    rg = rg.reshape(T, H + 2 * Hkv, d)
    dead = ~np.isfinite(rlse)
    assert np.array_equal(np.isneginf(lse), dead)
    assert (np.abs(lse[~dead] - rlse[~dead]) <= F32 * (1 + np.abs(rlse[~dead]))).all()
    tol_k, tol_v = np.zeros((T, Hkv, d)), np.zeros((T, Hkv, d))
    # codes below fp16's normal range: half a step of 2^-24, of rows whose largest is 1
    low = 2.0 ** -25 * np.abs(do).max()
    for h in range(H):
        g = h // (H // Hkv)
        # o: each probability rounded to fp16 (at least 2^-25 absolute, relative to a
        # largest one of 1 or more), then the result
        a = p[h] @ np.abs(v[:, g])
        tol_o = (HALF + F32) * (a + np.abs(ro[:, h])) + T * 2.0 ** -25 * np.abs(v).max()
        assert (np.abs(o[:, h] - ro[:, h]) <= tol_o).all(), ("o", h)
        # delta takes the rounded o; p and ds are rounded to fp16, the result to bf16
        dp = np.abs(do[:, h]) @ np.abs(v[:, g]).T
        ds = np.abs(p[h] * (do[:, h] @ v[:, g].T - (do[:, h] * ro[:, h]).sum(1)[:, None]))
        e = (HALF + F32) * ds + p[h] * (F32 * dp + (np.abs(do[:, h]) * tol_o).sum(1)[:, None])
        e = e / np.sqrt(d)
        tq = e @ np.abs(k[:, g]) + T * low / np.sqrt(d) * np.abs(k).max() + BF * np.abs(rg[:, h])
        assert (np.abs(got[:, h] - rg[:, h]) <= tq).all(), ("dq", h)
        tol_k[:, g] += e.T @ np.abs(q[:, h]) + T * low / np.sqrt(d) * np.abs(q).max()
        tol_v[:, g] += (HALF + F32) * (p[h].T @ np.abs(do[:, h])) + T * low
    assert (np.abs(got[:, H:H + Hkv] - rg[:, H:H + Hkv])
            <= tol_k + BF * np.abs(rg[:, H:H + Hkv])).all(), "dk"
    assert (np.abs(got[:, H + Hkv:] - rg[:, H + Hkv:])
            <= tol_v + BF * np.abs(rg[:, H + Hkv:])).all(), "dv"
    pad = ~op.visible(T, docs).any(1)
    assert not o[pad].any() and not got[pad].any()


@pytest.mark.parametrize("lengths,prefix,T", ROWS)
def test_index_and_targets(L, lengths, prefix, T):
    import torch
    idx = _index(L, lengths, prefix, T)
    docs = op.documents(lengths, prefix)
    words = idx.buf.cpu().numpy()
    cap = min(T, T // 128 + len(lengths))
    cap2 = min(T, T // 256 + len(lengths))
    for n, size, base, room in ((words[0], 128, 8, cap), (words[0], 128, 8 + 4 * cap, cap),
                                (words[1], 256, 8 + 8 * cap, cap2)):
        want = [(r, s, e, pe) for s, e, pe in docs for r in range(s, e, size)]
        assert n == len(want) <= room
        assert sorted(map(tuple, words[base:base + 4 * n].reshape(n, 4))) == sorted(want)
    # in order of falling work: the keys a query tile sees, the queries a key tile is seen by
    tiles = words[8:8 + 4 * words[0]].reshape(-1, 4)
    seen = np.minimum(tiles[:, 2], np.maximum(tiles[:, 0] + 128, tiles[:, 3])) - tiles[:, 1]
    assert (np.diff((seen + 127) // 128) <= 0).all()
    tiles = words[8 + 4 * cap:8 + 4 * (cap + words[0])].reshape(-1, 4)
    first = np.where(tiles[:, 0] < tiles[:, 3], tiles[:, 1], tiles[:, 0])
    assert (np.diff((tiles[:, 2] - first + 127) // 128) <= 0).all()
    assert words[2] == sum(lengths)
    pos, key_end, doc_end = words[8 + 4 * (2 * cap + cap2):].reshape(3, T)
    for s, e, pe in docs:
        for t in range(s, e):
            assert (pos[t], key_end[t], doc_end[t]) == (t - s, max(t + 1, pe), e)
    rng = np.random.default_rng(T)
    tok = rng.integers(0, 1000, T).astype(np.int32)
    for mask in (None, rng.integers(0, 2, T).astype(np.uint8)):
        want = op.targets(tok, docs, mask)
        y = torch.full((T,), -9, dtype=torch.int32, device="cuda")
        n = torch.full((1,), 5, dtype=torch.int32, device="cuda")
        m = None if mask is None else torch.from_numpy(mask).cuda()
        L.packed_targets(torch.from_numpy(tok).cuda(), idx, y, n, loss_mask=m)
        assert np.array_equal(y.cpu().numpy(), want) and n.item() == (want >= 0).sum()
        L.packed_targets(torch.from_numpy(tok).cuda(), idx, y, n,
                         loss_mask=None if m is None else m.bool(), accumulate=True)
        assert n.item() == 2 * (want >= 0).sum()
    assert L.lsq_device_status(clear=True) == 0


def test_tokens_below_zero_are_no_targets_and_are_not_counted(L):
    """Ids such as -100 mark what is not to be predicted: the mean is over the others."""
    import torch
    T, V, lengths = 300, 50, [120, 150]
    rng = np.random.default_rng(4)
    tok = rng.integers(0, V, T).astype(np.int32)
    tok[rng.random(T) < 0.4] = -100
    tok[5:8] = -1, -2, -2 ** 31
    idx = _index(L, lengths, None, T)
    want = op.targets(tok, op.documents(lengths))
    y = torch.full((T,), -9, dtype=torch.int32, device="cuda")
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.packed_targets(torch.from_numpy(tok).cuda(), idx, y, n)
    assert np.array_equal(y.cpu().numpy(), want) and n.item() == (want >= 0).sum() < 200
    x = rng.standard_normal((T, V)).astype(np.float32)
    rl, tot = torch.empty(T, device="cuda"), torch.empty(1, device="cuda")
    L.packed_cross_entropy(torch.from_numpy(x).cuda(), y, rl, tot, count=n)
    _, loss, _ = op.cross_entropy(x, want, None, int((want >= 0).sum()))
    # sums of 50 exponentials and of 160 rows in fp32
    assert abs(tot.item() - loss) <= 2.0 ** -16 * loss


def test_index_of_many_documents(L):
    """More documents than a pass of the scan takes, and a long row."""
    rng = np.random.default_rng(0)
    lengths = rng.integers(0, 40, 3000)
    T = int(lengths.sum()) + 11
    idx = _index(L, lengths.tolist(), None, T)
    words = idx.buf.cpu().numpy()
    ends = np.cumsum(lengths)
    starts = ends - lengths
    own = np.repeat(np.arange(3000), lengths)
    pos, key_end, doc_end = words[-3 * T:].reshape(3, T)
    n = T - 11
    assert np.array_equal(pos[:n], np.arange(n) - starts[own])
    assert np.array_equal(doc_end[:n], ends[own]) and (doc_end[n:] == n).all()
    assert words[0] == (lengths > 0).sum()


@pytest.mark.parametrize("n_docs", [32, 33, 1000, 1024, 1025])
def test_index_around_a_warp_and_a_block_of_documents(L, n_docs):
    """Short documents in a short row: the tiles outnumber a block's warps."""
    rng = np.random.default_rng(n_docs)
    lengths = np.where(rng.random(n_docs) < 0.9, 1, rng.integers(0, 300, n_docs))
    T = int(lengths.sum()) + 2
    words = _index(L, lengths.tolist(), None, T).buf.cpu().numpy()
    docs = op.documents(lengths.tolist(), None)
    cap, cap2 = min(T, T // 128 + n_docs), min(T, T // 256 + n_docs)
    for n, size, base in ((words[0], 128, 8), (words[0], 128, 8 + 4 * cap),
                          (words[1], 256, 8 + 8 * cap)):
        want = [(r, s, e, pe) for s, e, pe in docs for r in range(s, e, size)]
        got = words[base:base + 4 * n].reshape(n, 4)
        assert sorted(map(tuple, got)) == sorted(want)
        if n_docs <= 1024 and base == 8:
            seen = np.minimum(got[:, 2], got[:, 0] + 128) - got[:, 1]
            assert (np.diff((seen + 127) // 128) <= 0).all()
    pos, _, doc_end = words[-3 * T:].reshape(3, T)
    ends = np.cumsum(lengths)
    own = np.repeat(np.arange(n_docs), lengths)
    assert np.array_equal(pos[:T - 2], np.arange(T - 2) - (ends - lengths)[own])
    assert np.array_equal(doc_end[:T - 2], ends[own]) and (doc_end[T - 2:] == T - 2).all()


def test_a_new_index_is_a_row_of_padding(L):
    import torch
    H, Hkv, d, T = 4, 2, 64, 200
    qkv, dout = _inputs(T, H, Hkv, d, 1)
    o, lse, dqkv = _run(L, qkv.cuda(), dout.cuda(), L.PackedIndex(T, 3), H, Hkv)
    assert not o.any() and not dqkv.any() and torch.isneginf(lse).all()
    y, n = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    L.packed_targets(y, L.PackedIndex(T, 3), y.clone(), n)
    assert n.item() == 0


def test_index_bad_lengths_are_cut_and_latched(L):
    bad = L.LSQ_DEV_ERR_INDEX
    for lengths, prefix, T, total in (([5, -3, 4], None, 12, 9), ([5, 9], None, 10, 10),
                                      ([4, 4], [5, 0], 8, 8), ([4, 4], [-1, 0], 8, 8),
                                      ([8, 3], None, 8, 8)):
        idx = _index(L, lengths, prefix, T)
        assert idx.buf[2].item() == total
        assert L.lsq_device_status(clear=True) == bad


@pytest.mark.parametrize("H,Hkv,d", HEADS)
@pytest.mark.parametrize("lengths,prefix,T", ROWS)
def test_attention(L, lengths, prefix, T, H, Hkv, d):
    qkv, dout = _inputs(T, H, Hkv, d, seed=T + H)
    idx = _index(L, lengths, prefix, T)
    r = _run(L, qkv.cuda(), dout.cuda(), idx, H, Hkv)
    _check(qkv, dout, op.documents(lengths, prefix), H, Hkv, *r)


@pytest.mark.parametrize("H,Hkv,d", [(4, 2, 128), (3, 1, 64)])
def test_attention_large_scores_and_extreme_gradients(L, H, Hkv, d):
    """Scores of some hundreds (one key takes all), and gradients far below and above
    what fp16 holds, of different size from row to row."""
    import torch
    T, lengths = 300, [260, 40]
    idx = _index(L, lengths, None, T)
    docs = op.documents(lengths)
    qkv, dout = _inputs(T, H, Hkv, d, 3, grad=1.0)
    qkv[:, :(H + Hkv) * d] *= 6
    for scale in (1e-30, 1e30):
        g = (dout.float() * scale).bfloat16()
        o, lse, dqkv = _run(L, qkv.cuda(), g.cuda(), idx, H, Hkv)
        ref = op.attention_bwd(qkv.float().numpy(), H, Hkv, docs, g.float().numpy())
        got = dqkv.float().cpu().numpy()
        # scores of size s carry an error of s 2^-22 or so; q k / sqrt d is below 2^10
        assert np.abs(got - ref).max() <= 2.0 ** -7 * np.abs(ref).max()
    zero = torch.zeros_like(dout)
    assert not _run(L, qkv.cuda(), zero.cuda(), idx, H, Hkv)[2].any()


@pytest.mark.parametrize("H,Hkv,d", [(4, 2, 64), (3, 3, 128)])
def test_nothing_crosses_a_document(L, H, Hkv, d):
    """Infinities and NaN in one document and in the padding leave the others' results
    bit for bit as they are."""
    import torch
    lengths, prefix, T = [70, 130, 90, 20], [10, 60, 0, 20], 330
    idx = _index(L, lengths, prefix, T)
    qkv, dout = _inputs(T, H, Hkv, d, 5)
    clean = _run(L, qkv.cuda(), dout.cuda(), idx, H, Hkv)
    for bad in (float("nan"), float("inf")):
        q2, g2 = qkv.clone(), dout.clone()
        for a, e in ((70, 200), (310, 330)):
            q2[a:e] = bad
            g2[a:e] = bad
        qc, gc = q2.cuda(), g2.cuda()
        o = torch.empty_like(clean[0])
        lse, dqkv = torch.empty_like(clean[1]), torch.empty_like(clean[2])
        ws = torch.empty(L.packed_attention_workspace_bytes(T, H, Hkv, d), dtype=torch.uint8,
                         device="cuda")
        L.packed_attention_fwd(qc, idx, H, Hkv, o, lse)
        L.packed_attention_bwd(qc, idx, o, lse, gc, H, Hkv, dqkv, ws)
        torch.cuda.synchronize()
        assert L.lsq_device_status(clear=True) == L.LSQ_DEV_ERR_NONFINITE
        keep = torch.ones(T, dtype=torch.bool)
        keep[70:200] = False
        keep = keep.cuda()
        assert torch.equal(o[keep], clean[0][keep])
        assert torch.equal(lse[:, keep], clean[1][:, keep])
        assert torch.equal(dqkv[keep], clean[2][keep])


@pytest.mark.parametrize("H,Hkv,d", [(2, 1, 64), (1, 1, 128), (4, 1, 128)])
@pytest.mark.parametrize("vstd,outlier", [(1.0, 1), (0.03, 256), (0.003, 1), (0.0003, 1),
                                          (1.0, 4096), (1e-6, 64), (300.0, 1)])
def test_gradients_of_a_long_diffuse_document(L, H, Hkv, d, vstd, outlier):
    """Thousands of small probabilities, small or large v, one query whose gradient is far
    above the others': no row of dq, dk and dv may lose its small parts in fp16.  Of each
    row's norm: the result's rounding to bf16 (2^-8), and those of P, dS and dO's products to
    fp16, 2^-11 each, of terms that add up as the terms themselves do.  delta takes o rounded
    to fp16, off by 2^-11 |dO| |o| or 2^-25 |dO| at most, whatever is left of dP - delta."""
    import torch
    lengths, T = [700, 4096, 100], 4900
    g = torch.Generator().manual_seed(int(1e6 * vstd) + outlier)
    qkv = torch.randn(T, H + 2 * Hkv, d, generator=g)
    qkv[:, :H + Hkv] *= 0.3
    qkv[:, H + Hkv:] *= vstd
    dout = torch.randn(T, H, d, generator=g) * 1e-5
    dout[2900] *= outlier              # in the middle of the long document
    qkv, dout = qkv.reshape(T, -1).half().cuda(), dout.reshape(T, -1).bfloat16().cuda()
    o, lse, dqkv = _run(L, qkv, dout, _index(L, lengths, None, T), H, Hkv)
    got = dqkv.double().view(T, H + 2 * Hkv, d)
    x, do = qkv.double().view(T, H + 2 * Hkv, d), dout.double().view(T, H, d)
    tol, h11 = 2.0 ** -8 + 3 * 2.0 ** -11, 2.0 ** -11 + F32
    for s, e, _ in op.documents(lengths):
        dk, dv = (torch.zeros(e - s, Hkv, d, dtype=torch.float64, device="cuda") for _ in "kv")
        low_k = torch.zeros(e - s, Hkv, dtype=torch.float64, device="cuda")
        for h in range(H):
            n = h // (H // Hkv)
            q, k, v = x[s:e, h], x[s:e, H + n], x[s:e, H + Hkv + n]
            p = torch.softmax((q @ k.T / d ** 0.5).masked_fill(
                torch.ones(e - s, e - s, dtype=torch.bool, device="cuda").triu(1), -float("inf")), 1)
            ro = p @ v
            ds = p * (do[s:e, h] @ v.T - (do[s:e, h] * ro).sum(1)[:, None]) / d ** 0.5
            dq = ds @ k
            off = p * ((do[s:e, h].abs() * (h11 * ro.abs() + 2.0 ** -25)).sum(1) / d ** 0.5)[:, None]
            err = (got[s:e, h] - dq).norm(dim=1)
            assert (err <= tol * dq.norm(dim=1) + off @ k.norm(dim=1)).all(), ("dq", h, s)
            dk[:, n] += ds.T @ q
            dv[:, n] += p.T @ do[s:e, h]
            low_k[:, n] += off.T @ q.norm(dim=1)
        err = (got[s:e, H:H + Hkv] - dk).norm(dim=2)
        assert (err <= tol * dk.norm(dim=2) + low_k).all(), ("dk", s)
        err = (got[s:e, H + Hkv:] - dv).norm(dim=2)
        assert (err <= tol * dv.norm(dim=2)).all(), ("dv", s)


def test_large_values_keep_finite_gradients(L):
    """Rows of v up to fp16's largest numbers: the score gradients are scaled before they are
    rounded, and nothing is latched."""
    import torch
    H, Hkv, d, T, lengths = 4, 2, 64, 300, [200, 90]
    qkv, dout = _inputs(T, H, Hkv, d, 6)
    qkv[:, (H + Hkv) * d:] = (qkv[:, (H + Hkv) * d:].float() * 12000).clamp(-65504, 65504).half()
    _, _, dqkv = _run(L, qkv.cuda(), dout.cuda(), _index(L, lengths, None, T), H, Hkv)
    want = op.attention_bwd(qkv.float().numpy(), H, Hkv, op.documents(lengths), dout.float().numpy())
    got = dqkv.float().cpu().numpy()
    assert np.isfinite(got).all()
    for lo, hi in ((0, H * d), (H * d, (H + Hkv) * d), ((H + Hkv) * d, None)):
        a, b = got[:, lo:hi], want[:, lo:hi]
        # the worst row's roundings of 300 terms of one sign, 2^-11 each, then bf16's
        assert np.abs(a - b).max() <= 2.0 ** -7 * np.abs(b).max()


def test_attention_is_deterministic_on_any_stream_and_in_a_graph(L):
    import torch
    H, Hkv, d, T, lengths = 8, 2, 64, 500, [300, 190]
    idx = _index(L, lengths, None, T)
    qkv, dout = (x.cuda() for x in _inputs(T, H, Hkv, d, 8))
    a = _run(L, qkv, dout, idx, H, Hkv)
    b = _run(L, qkv, dout, idx, H, Hkv, ws_fill=0)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c = _run(L, qkv, dout, idx, H, Hkv)
    assert all(torch.equal(x, y) for x, y in zip(a, c))
    # captured with its index, replayed on other documents and other values
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out = [torch.empty_like(x) for x in a]
    ws = torch.empty(L.packed_attention_workspace_bytes(T, H, Hkv, d), dtype=torch.uint8,
                     device="cuda")

    def step():
        L.packed_index(lens, idx)
        L.packed_attention_fwd(qkv, idx, H, Hkv, out[0], out[1])
        L.packed_attention_bwd(qkv, idx, out[0], out[1], dout, H, Hkv, out[2], ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, out))
    q2, g2 = (x.cuda() for x in _inputs(T, H, Hkv, d, 9))
    qkv.copy_(q2)
    dout.copy_(g2)
    lens.copy_(torch.tensor([0, 450], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    _check(q2.cpu(), g2.cpu(), op.documents([0, 450]), H, Hkv, *out)


LOSS = [(1, 1), (1, 2), (3, 7), (5, 8), (4, 1001), (6, 4096), (2, 5003), (3, 40000), (2, 131075),
        (2, 460003)]


@pytest.mark.parametrize("H,Hkv,d", [(4, 2, 64), (4, 1, 128), (3, 1, 128)])
def test_attention_problems_that_follow_one_another_in_the_same_memory(L, H, Hkv, d):
    """Two rows alternate over one index, workspace and set of inputs and outputs, with
    fewer CTAs than SMs: nothing of the row before may be met again in a cache."""
    import torch
    T = 300
    rows = [([100, 200, 0, 0], [0, 50, 0, 0]), ([37, 1, 200, 62], None)]
    data = [tuple(t.cuda() for t in _inputs(T, H, Hkv, d, seed=9 + i)) for i in range(2)]
    lens = [torch.tensor(a, dtype=torch.int32, device="cuda") for a, _ in rows]
    pre = [None if b is None else torch.tensor(b, dtype=torch.int32, device="cuda")
           for _, b in rows]
    want = [_run(L, *data[i], _index(L, *rows[i], T), H, Hkv) for i in range(2)]
    idx = L.PackedIndex(T, 4)
    qkv, dout = (torch.empty_like(t) for t in data[0])
    o, lse, dqkv = (torch.empty_like(t) for t in want[0])
    ws = torch.empty(L.packed_attention_workspace_bytes(T, H, Hkv, d), dtype=torch.uint8,
                     device="cuda")
    same = torch.ones(1, dtype=torch.bool, device="cuda")
    for k in range(40):
        i = k & 1
        qkv.copy_(data[i][0])
        dout.copy_(data[i][1])
        L.packed_index(lens[i], idx, prefix=pre[i])
        L.packed_attention_fwd(qkv, idx, H, Hkv, o, lse)
        L.packed_attention_bwd(qkv, idx, o, lse, dout, H, Hkv, dqkv, ws)
        for got, ref in zip((o, lse, dqkv), want[i]):
            same &= (got == ref).all()
    assert same.item() and L.lsq_device_status(clear=True) == 0


@pytest.mark.parametrize("T,V", LOSS)
@pytest.mark.parametrize("form", ["plain", "weighted", "none"])
def test_cross_entropy(L, T, V, form):
    import torch
    rng = np.random.default_rng(T * V)
    x = (rng.standard_normal((T, V)) * 3).astype(np.float32)
    y = rng.integers(0, V, T).astype(np.int32)
    y[rng.random(T) < 0.3] = -1
    y[0] = -100 if form == "none" else V - 1
    if form == "none":
        y[:] = -1
    w = rng.random(T).astype(np.float32) if form == "weighted" else None
    n = int((y >= 0).sum()) if form != "weighted" else None
    if V > 20:
        x[0, 3:9] = -np.inf         # excluded words
        x[y < 0] = np.nan           # rows without a target are not read
    row, loss, grad = op.cross_entropy(np.nan_to_num(x, nan=0.0, neginf=-1e30), y, w, n)
    dl = torch.full((T, V), float("nan"), dtype=torch.bfloat16, device="cuda")
    rl = torch.full((T,), float("nan"), device="cuda")
    tot = torch.full((1,), 2.5, device="cuda")
    kw = dict(weight=None if w is None else torch.from_numpy(w).cuda(),
              count=None if n is None else torch.tensor([n], dtype=torch.int32, device="cuda"))
    xd, yd = torch.from_numpy(x).cuda(), torch.from_numpy(y).cuda()
    L.packed_cross_entropy(xd, yd, rl, tot, dlogits=dl, **kw)
    # arguments of exp2 below 64 in magnitude: 2^-17 relative; sums of V terms, V / 128
    # of them in a row
    tol = 2.0 ** -16 + V / 128 * 2.0 ** -24
    assert (np.abs(rl.cpu().numpy() - row) <= tol * (1 + np.abs(row))).all()
    c = np.zeros(T)
    c[y >= 0] = (1.0 if w is None else w[y >= 0]) / (1 if n is None else max(n, 1))
    assert abs(tot.item() - loss) <= 2 * tol * (1 + abs(loss))
    err = np.abs(dl.float().cpu().numpy() - grad)
    assert (err <= BF * np.abs(grad) + tol * c[:, None]).all()
    only = torch.empty_like(rl)
    L.packed_cross_entropy(xd, yd, only, tot, accumulate=True, **kw)
    assert torch.equal(only, rl)
    assert abs(tot.item() - 2 * loss) <= 4 * tol * (1 + abs(loss))
    assert L.lsq_device_status(clear=True) == 0


def test_cross_entropy_target_beyond_the_vocabulary(L):
    import torch
    x = torch.randn(3, 50, device="cuda")
    y = torch.tensor([1, 50, 7], dtype=torch.int32, device="cuda")
    rl, tot = torch.empty(3, device="cuda"), torch.empty(1, device="cuda")
    dl = torch.empty(3, 50, dtype=torch.bfloat16, device="cuda")
    L.packed_cross_entropy(x, y, rl, tot, dlogits=dl)
    assert rl[1].item() == 0 and not dl[1].any() and dl[0].any()
    assert abs(tot.item() - (rl[0] + rl[2]).item()) < 1e-5
    assert L.lsq_device_status(clear=True) == L.LSQ_DEV_ERR_INDEX


def test_cross_entropy_not_finite_rows_are_the_formulas(L):
    import torch
    x = torch.randn(3, 300, device="cuda")
    x[0] = -float("inf")
    x[1, 5] = float("inf")
    x[2, 9] = -float("inf")
    y = torch.tensor([4, 5, 9], dtype=torch.int32, device="cuda")
    rl, tot = torch.empty(3, device="cuda"), torch.empty(1, device="cuda")
    L.packed_cross_entropy(x, y, rl, tot)
    assert torch.isnan(rl[0]) and torch.isnan(rl[1]) and rl[2].item() == float("inf")


@pytest.mark.parametrize("T,V", [(4, 1), (4, 7), (5, 300), (5, 1001), (5, 40003), (4, 131075),
                                 (4, 460003)])
def test_cross_entropy_a_nan_anywhere_reaches_the_whole_row(L, T, V):
    """Also among the few logits before and behind those that are taken eight at a time, and
    in a row that holds nothing else; the other rows do not change."""
    import torch
    nan, inf = float("nan"), float("inf")
    g = torch.Generator().manual_seed(V)
    clean = torch.randn(T, V, generator=g).cuda()
    y = torch.full((T,), V // 2, dtype=torch.int32, device="cuda")

    def run(x):
        rl, tot = torch.empty(T, device="cuda"), torch.empty(1, device="cuda")
        dl = torch.empty(T, V, dtype=torch.bfloat16, device="cuda")
        L.packed_cross_entropy(x, y, rl, tot, dlogits=dl)
        return rl, tot, dl
    rl0, _, dl0 = run(clean)
    for row in range(T):
        for at in sorted({0, 1, 7, 8, V // 2, V - 9, V - 8, V - 2, V - 1} & set(range(V))):
            for rest in (False, True):
                x = clean.clone()
                if rest:
                    x[row] = -inf       # nothing finite to take a maximum of
                x[row, at] = nan
                rl, tot, dl = run(x)
                assert torch.isnan(rl[row]) and torch.isnan(tot[0]), (row, at, rest)
                assert torch.isnan(dl[row]).all(), (row, at, rest)
                keep = torch.arange(T, device="cuda") != row
                assert torch.equal(rl[keep], rl0[keep]) and torch.equal(dl[keep], dl0[keep])
    assert L.lsq_device_status(clear=True) == 0


def test_attention_of_many_short_documents(L):
    """More work items than a GPU has SMs, each with a cleared tail: every CTA takes
    several in turn."""
    lengths = [1 + (i * 7) % 30 for i in range(60)]
    T, H, Hkv, d = sum(lengths) + 5, 8, 2, 64
    qkv, dout = _inputs(T, H, Hkv, d, seed=2)
    idx = _index(L, lengths, None, T)
    r = _run(L, qkv.cuda(), dout.cuda(), idx, H, Hkv)
    _check(qkv, dout, op.documents(lengths), H, Hkv, *r)


@pytest.mark.parametrize("prefix", [False, True])
def test_attention_of_a_long_row(L, prefix):
    """Many items of many steps a CTA: against plain torch in fp32, document by document."""
    import torch
    rng = np.random.default_rng(1)
    H, Hkv, d, lengths = 16, 2, 128, []
    while sum(lengths) < 9000:
        lengths.append(int(np.exp(rng.uniform(np.log(32), np.log(2048)))))
    T = sum(lengths) + 100
    pre = [int(rng.integers(0, n + 1)) for n in lengths] if prefix else None
    qkv, dout = (x.cuda() for x in _inputs(T, H, Hkv, d, 4))
    idx = _index(L, lengths, pre, T)
    o, lse, dqkv = _run(L, qkv, dout, idx, H, Hkv)
    # error of a row of n terms against its largest value: roundings of 2^-11 (p) and
    # 2^-8 (bf16) relative to sums that are never larger than ~sqrt(n) times the result
    for k, (s, e, pe) in enumerate(op.documents(lengths, pre)):
        x = qkv[s:e].float().view(e - s, H + 2 * Hkv, d).permute(1, 0, 2)
        q, kk, v = x[:H], x[H:H + Hkv].repeat_interleave(8, 0), x[H + Hkv:].repeat_interleave(8, 0)
        at = torch.arange(e - s, device="cuda")
        see = (at[None] <= at[:, None]) | (at[None] < pe - s)
        sc = (q @ kk.transpose(1, 2) / d ** 0.5).masked_fill(~see, -float("inf"))
        p = sc.softmax(-1)
        ro = p @ v
        do = dout[s:e].float().view(e - s, H, d).permute(1, 0, 2)
        ds = p * (do @ v.transpose(1, 2) - (do * ro).sum(-1, keepdim=True)) / d ** 0.5
        dq, dk = ds @ kk, (ds.transpose(1, 2) @ q).view(Hkv, 8, e - s, d).sum(1)
        dv = (p.transpose(1, 2) @ do).view(Hkv, 8, e - s, d).sum(1)
        ref = torch.cat([dq, dk, dv]).permute(1, 0, 2).reshape(e - s, -1)
        assert (lse[:, s:e] - sc.logsumexp(-1)).abs().max() <= 1e-4, k
        for got, want, tol in ((o[s:e].float(), ro.permute(1, 0, 2).reshape(e - s, -1), 2.0 ** -9),
                               (dqkv[s:e].float(), ref, 2.0 ** -7)):
            assert (got - want).norm() <= tol * want.norm(), k
            assert (got - want).abs().max() <= 4 * tol * want.abs().max(), k
