"""The packed operators together, as a fine-tuning step uses them: a decoder layer and a
streamed stack step on packed rows (index, positions, attention inside documents, targets,
cross-entropy, AdamW with an 8-bit state) against the fp64 oracle run document by
document.  Tolerances are the stack's: loss 1e-3 relative, activations and gradients 2e-2
(gpu_util.check_stack_grad); the optimiser's state bit for bit."""
import numpy as np
import pytest

from oracle import model as om
from oracle import packed as op
from layer_streamed_qlora_nf4_b200 import synth
from test_gpu_layer import _device_layer, _oracle_params
from test_gpu_stack import Stack

pytestmark = pytest.mark.gpu
TOL = 2e-2

ROWS = [[40, 1, 0, 55], [64, 20, 9, 3]]      # documents of two rows of 100 tokens
PROMPTS = [[13, 0, 0, 55], [0, 20, 1, 2]]
T = 100


@pytest.fixture(scope="module")
def L():
    from layer_streamed_qlora_nf4_b200 import lib
    lib.load()
    return lib


@pytest.fixture(scope="module")
def small(L):
    return Stack(L, synth.SMALL, 5)


class _Prompt:
    """While active, the oracle's attention reads the first `n` tokens in both directions."""

    def __init__(self, n):
        self.n, self.kept = n, (om.attention, om.attention_bwd)

    @staticmethod
    def _flat(q, k, v):
        return np.concatenate([x.reshape(len(x), -1) for x in (q, k, v)], 1)

    def __enter__(self):
        def fwd(q, k, v):
            docs = [(0, len(q), self.n)]
            return op.attention_fwd(self._flat(q, k, v), q.shape[1], k.shape[1], docs)[:2]

        def bwd(do, q, k, v):
            docs, (S, H, d), Hkv = [(0, len(q), self.n)], q.shape, k.shape[1]
            g = op.attention_bwd(self._flat(q, k, v), H, Hkv, docs, do).reshape(S, H + 2 * Hkv, d)
            return g[:, :H], g[:, H:H + Hkv], g[:, H + Hkv:]
        om.attention, om.attention_bwd = fwd, bwd

    def __exit__(self, *exc):
        om.attention, om.attention_bwd = self.kept


@pytest.mark.parametrize("prompts", [False, True])
def test_layer(L, prompts):
    import torch
    from gpu_util import dev, normwise_err, workspace
    from layer_streamed_qlora_nf4_b200 import pack
    cfg = synth.SMALL
    lw = synth.layer_weights(3, cfg)
    x = synth.bf16_bits_to_f32(synth.activations(4, T, cfg["hidden"]))
    dout = synth.normal_f32(synth.rng(5), (T, cfg["hidden"]), 1.0)
    lens, pre = ROWS[0], PROMPTS[0] if prompts else [0] * 4
    dout[sum(lens):] = 0                       # padding has no loss
    blob, lora = _device_layer(L, cfg, lw)
    idx = L.PackedIndex(T, len(lens))
    L.packed_index(torch.tensor(lens, dtype=torch.int32, device="cuda"), idx,
                   prefix=torch.tensor(pre, dtype=torch.int32, device="cuda"))
    ws = workspace(L.decoder_layer_workspace_bytes(cfg, 1, T))
    y, dx = torch.empty(T, cfg["hidden"], device="cuda"), torch.empty(T, cfg["hidden"], device="cuda")
    grad = torch.full_like(lora, float("nan"))
    L.decoder_layer_packed_fwd(cfg, blob, lora, dev(x), idx, y, ws)
    L.decoder_layer_packed_bwd(cfg, blob, lora, dev(x), dev(dout), idx, dx, grad, ws)
    torch.cuda.synchronize()
    assert L.lsq_device_status(clear=True) == 0
    p = _oracle_params(lw, cfg)
    total = None
    for (s, e, pe) in op.documents(lens, pre):
        if e == s:
            continue
        with _Prompt(pe - s):
            ry, _ = om.decoder_layer_fwd(p, x[s:e], cfg, e - s)
            rdx, rg = om.decoder_layer_bwd(p, x[s:e], dout[s:e], cfg, e - s)
        assert normwise_err(y[s:e].cpu().numpy(), ry) <= TOL
        assert normwise_err(dx[s:e].cpu().numpy(), rdx) <= TOL
        if total is None:
            total = rg
        else:
            total = {n: tuple(a + b for a, b in zip(total[n], rg[n])) for n in rg}
    views = pack.lora_views(cfg, grad)
    for n in synth.PROJ:
        for k in (0, 1):
            assert normwise_err(views[n][k].cpu().numpy(), total[n][k]) <= TOL, (n, k)


def _batch(seed, prompts, masked):
    import torch
    rng = np.random.default_rng(seed)
    tokens = rng.integers(0, synth.SMALL["vocab"], (2, T)).astype(np.int32)
    mask = rng.integers(0, 2, (2, T)).astype(np.uint8) if masked else None
    d = dict(tokens=torch.from_numpy(tokens).cuda(),
             lengths=torch.tensor(ROWS, dtype=torch.int32, device="cuda"),
             prefix=torch.tensor(PROMPTS, dtype=torch.int32, device="cuda") if prompts else None,
             loss_mask=torch.from_numpy(mask).cuda() if masked else None)
    return tokens, mask, d


def _run(L, st, h, d, opt=None, step=1, lora=None, grad=None):
    import torch
    from gpu_util import workspace
    ws = workspace(L.stream_stack_packed_workspace_bytes(st.cfg, T, 4))
    lora = st.lora.clone() if lora is None else lora
    grad = torch.full_like(lora, float("nan")) if grad is None else grad
    logits = torch.empty(T, st.cfg["vocab"], device="cuda")
    loss = L.stream_stack_packed_step(h, d["tokens"], d["lengths"], st.emb, st.head, st.gf, lora,
                                      grad, ws, prefix=d["prefix"], loss_mask=d["loss_mask"],
                                      opt=opt, step=step, logits_out=logits)
    return loss, logits, grad, lora


@pytest.mark.parametrize("prompts,masked", [(False, False), (True, True)])
def test_step_matches_oracle(L, small, prompts, masked):
    from gpu_util import check_stack_grad, normwise_err
    from layer_streamed_qlora_nf4_b200 import pack
    tokens, mask, d = _batch(11, prompts, masked)
    h = small.handle(L, resident=False)
    loss, logits, grad, _ = _run(L, small, h, d)
    h.close()
    cfg, layers = small.cfg, small.oracle_layers()
    emb, head, gf = (synth.bf16_bits_to_f32(b) for b in (small.emb_bits, small.head_bits, small.gf_bits))
    rows = [op.documents(r, p if prompts else None) for r, p in zip(ROWS, PROMPTS)]
    ys = [op.targets(tokens[m], rows[m], None if mask is None else mask[m]) for m in (0, 1)]
    n = sum(int((y >= 0).sum()) for y in ys)
    rloss, total = 0.0, None
    for m in (0, 1):
        for s, e, pe in rows[m]:
            if e == s:
                continue
            with _Prompt(pe - s):
                lg, c = om.stack_forward(layers, emb, head, gf, tokens[m][None, s:e], cfg)
                _, part, dl = op.cross_entropy(lg.reshape(e - s, -1), ys[m][s:e], None, n)
                rloss += part
                dh = om.rmsnorm_bwd(dl @ head.astype(np.float64), c["h"], gf, cfg["rms_eps"])
                grads = [None] * len(layers)
                for i in range(len(layers) - 1, -1, -1):
                    dh, grads[i] = om.decoder_layer_bwd(layers[i], c["xs"][i], dh, cfg, e - s)
            if m == 1:
                assert normwise_err(logits[s:e].cpu().numpy(), lg.reshape(e - s, -1)) <= TOL
            total = grads if total is None else [
                {k: tuple(a + b for a, b in zip(t[k], g[k])) for k in g} for t, g in zip(total, grads)]
    assert abs(loss - rloss) <= 1e-3 * abs(rloss), (loss, rloss)
    nf = L.lsq_lora_layout_get(cfg).floats_per_layer
    for i in range(cfg["n_layers"]):
        views = pack.lora_views(cfg, grad[i * nf:(i + 1) * nf])
        for name in synth.PROJ:
            for k in (0, 1):
                check_stack_grad(views[name][k].cpu().numpy(), total[i][name][k], name, (i, k))


def _tensors(L, cfg, buf):
    from layer_streamed_qlora_nf4_b200 import pack
    nf = L.lsq_lora_layout_get(cfg).floats_per_layer
    return [x for i in range(cfg["n_layers"])
            for v in pack.lora_views(cfg, buf[i * nf:(i + 1) * nf]).values() for x in v]


def _optimiser(L, cfg, lora, grad):
    """8-bit AdamW over every A and B, the B factors at twice the rate and without decay."""
    import torch
    p, g = _tensors(L, cfg, lora), _tensors(L, cfg, grad)
    m = [torch.zeros(x.numel(), dtype=torch.int8, device="cuda") for x in p]
    v = [torch.zeros(x.numel(), dtype=torch.uint8, device="cuda") for x in p]
    ms, vs = ([torch.zeros(L.adamw_scale_floats(x.numel()), device="cuda") for x in p] for _ in "mv")
    lr, wd = [2e-4, 4e-4] * (len(p) // 2), [0.01, 0.0] * (len(p) // 2)
    return L.AdamWMulti(p, g, m, v, lr, wd, m_scale=ms, v_scale=vs), (p, g, m, v, ms, vs, lr, wd)


def test_steps_with_the_8bit_optimiser(L, small):
    """Three steps on different rows: the state and parameters are those of the oracle's
    update of the step's own gradients, and streamed equals resident bit for bit."""
    import torch
    runs = []
    for resident in (False, True):
        h = small.handle(L, resident)
        lora = small.lora.clone()
        grad = torch.full_like(lora, float("nan"))
        opt, parts = _optimiser(L, small.cfg, lora, grad)
        kept = []
        state = [(np.zeros(x.numel(), np.int8), np.zeros(x.numel(), np.uint8), None, None)
                 for x in parts[0]]
        for step in (1, 2, 3):
            before = [x.cpu().numpy().reshape(-1) for x in parts[0]]
            _, _, d = _batch(20 + step, step == 2, step > 1)
            loss, logits, _, _ = _run(L, small, h, d, opt=opt, step=step, lora=lora, grad=grad)
            kept += [torch.tensor(loss), logits.clone(), grad.clone(), lora.clone()]
            if resident:
                continue
            for i in range(len(parts[0])):
                mc, vc, ms, vs = state[i]
                g = parts[1][i].cpu().numpy().reshape(-1)
                m = np.zeros(len(g), np.float32) if ms is None else op.decode(mc, ms)
                v = np.zeros(len(g), np.float32) if vs is None else op.decode(vc, vs)
                p, m, v = op.adamw(before[i], g, m, v, step, parts[6][i], parts[7][i])
                (mc, ms), (vc, vs) = op.encode(m, True), op.encode(v, False)
                state[i] = mc, vc, ms, vs
                for got, want in zip(parts[2:6], state[i]):
                    assert np.array_equal(got[i].cpu().numpy(), want), (step, i)
                # a rounding of p and an update of a few lr, as in test_gpu_adamw_multi
                tol = 2.0 ** -23 * np.abs(p) + 2.0 ** -20 * 10 * parts[6][i]
                e = np.abs(parts[0][i].cpu().numpy().reshape(-1) - p)
                assert (e <= tol).all(), (step, i, (e / tol).max())
        runs.append(kept)
        h.close()
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    assert L.lsq_device_status(clear=True) == 0


def test_step_without_targets(L, small):
    """Nothing to train on: loss 0 and zero gradients, not NaN."""
    import torch
    _, _, d = _batch(31, False, False)
    d["loss_mask"] = torch.zeros(2, T, dtype=torch.bool, device="cuda")
    h = small.handle(L, resident=True)
    loss, _, grad, _ = _run(L, small, h, d)
    h.close()
    assert loss == 0.0 and not grad.any()


@pytest.mark.parametrize("what", ["length", "prompt", "token"])
def test_a_step_with_bad_documents_updates_nothing(L, small, what):
    """Parameters, moments and scales are bit for bit as before the refused step, and the step
    that follows with sound documents is the one that would have been without it."""
    import torch
    runs = []
    for bad_first in (False, True):
        h = small.handle(L, resident=False)
        lora = small.lora.clone()
        grad = torch.full_like(lora, float("nan"))
        opt, parts = _optimiser(L, small.cfg, lora, grad)
        _run(L, small, h, _batch(21, True, False)[2], opt=opt, step=1, lora=lora, grad=grad)

        def state():
            return [t.clone() for k in (0, 2, 3, 4, 5) for t in parts[k]]
        if bad_first:
            _, _, d = _batch(22, True, False)
            if what == "length":
                d["lengths"][1, 1] = 60
            elif what == "prompt":
                d["prefix"][0, 0] = 41
            else:
                d["tokens"][1, 30] = small.cfg["vocab"]   # a target: this document has no prompt
            before = state()
            with pytest.raises(L.LsqError) as e:
                _run(L, small, h, d, opt=opt, step=2, lora=lora, grad=grad)
            assert e.value.code == L.LSQ_ERR_DEVICE
            assert all(torch.equal(a, b) for a, b in zip(before, state()))
            assert L.lsq_device_status(clear=True) == L.LSQ_DEV_ERR_INDEX
        loss, _, _, _ = _run(L, small, h, _batch(22, True, False)[2], opt=opt, step=2, lora=lora,
                             grad=grad)
        runs.append([torch.tensor(loss)] + state())
        h.close()
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_step_refusals(L, small):
    import torch
    _, _, d = _batch(1, False, False)
    h = small.handle(L, resident=True)
    d["lengths"][0, 0] = 99                     # documents longer than the row
    with pytest.raises(L.LsqError) as e:
        _run(L, small, h, d)
    assert e.value.code == L.LSQ_ERR_DEVICE
    assert L.lsq_device_status(clear=True) == L.LSQ_DEV_ERR_INDEX
    _, _, d = _batch(1, False, False)
    lora = small.lora.clone()
    grad = torch.empty_like(lora)
    opt, _ = _optimiser(L, small.cfg, lora, grad)
    with pytest.raises(L.LsqError) as e:
        _run(L, small, h, d, opt=opt, step=0, lora=lora, grad=grad)
    assert e.value.code == L.LSQ_ERR_SHAPE
    ws = torch.empty(1024, dtype=torch.uint8, device="cuda")
    args = (h, d["tokens"], d["lengths"], small.emb, small.head, small.gf, lora, grad, ws)
    with pytest.raises(L.LsqError) as e:
        L.stream_stack_packed_step(*args)
    assert e.value.code == L.LSQ_ERR_WORKSPACE
    with pytest.raises(ValueError):
        L.stream_stack_packed_step(h, d["tokens"][0], *args[2:])
    with pytest.raises(ValueError):
        L.stream_stack_packed_step(*args, loss_mask=torch.zeros(2, 9, dtype=torch.bool, device="cuda"))
    h.close()
