"""Packed layers and steps in the forms that test_gpu_packed_step.py's small model does not
reach: heads of 128, groups of one, three and four heads, bf16 weights, 8-bit absmax, rank 64;
few long documents and many short ones (dK and dV of a kv head in several shares and in one, the
rotation of k undone in either); a head in several chunks.  Against the fp64 oracle document by
document, at the stack's tolerances."""
import numpy as np
import pytest

from oracle import model as om
from oracle import packed as op
from layer_streamed_qlora_nf4_b200 import synth
from test_gpu_layer import _device_layer, _oracle_params
from test_gpu_packed_step import TOL, _Prompt
from test_gpu_stack import Stack

pytestmark = pytest.mark.gpu

CFGS = {
    "d64": synth.SMALL,
    "d128, groups of 2": dict(synth.SMALL, n_heads=4, n_kv_heads=2, head_dim=128),
    "d128, a group of 3, absmax of 8 bits": dict(synth.SMALL, n_heads=3, n_kv_heads=1,
                                                 head_dim=128, absmax_bits=8),
    "d128, single heads": dict(synth.SMALL, n_heads=4, n_kv_heads=4, head_dim=128),
    "d128, a group of 4, bf16 weights, rank 64": dict(synth.SMALL, n_heads=4, n_kv_heads=1,
                                                      head_dim=128, weight_bits=16, lora_r=64),
}
ROWS = [
    # lengths, prompts, tokens
    ([290], [0], 300),
    ([150, 131], [40, 131], 290),
    ([20, 17, 1, 30, 0, 25, 9, 12, 3, 8], [3, 0, 1, 30, 0, 0, 8, 0, 0, 5], 131),
]


@pytest.fixture(scope="module")
def L():
    from layer_streamed_qlora_nf4_b200 import lib
    lib.load()
    return lib


@pytest.mark.parametrize("lens,pre,T", ROWS)
@pytest.mark.parametrize("form", list(CFGS))
def test_layer(L, form, lens, pre, T):
    import torch
    from gpu_util import dev, normwise_err, workspace
    from layer_streamed_qlora_nf4_b200 import pack
    cfg = CFGS[form]
    lw = synth.layer_weights(3, cfg)
    x = synth.bf16_bits_to_f32(synth.activations(4, T, cfg["hidden"]))
    dout = synth.normal_f32(synth.rng(5), (T, cfg["hidden"]), 1.0)
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
    p, total = _oracle_params(lw, cfg), None
    for s, e, pe in op.documents(lens, pre):
        if e == s:
            continue
        with _Prompt(pe - s):
            ry, _ = om.decoder_layer_fwd(p, x[s:e], cfg, e - s)
            rdx, rg = om.decoder_layer_bwd(p, x[s:e], dout[s:e], cfg, e - s)
        assert normwise_err(y[s:e].cpu().numpy(), ry) <= TOL
        assert normwise_err(dx[s:e].cpu().numpy(), rdx) <= TOL
        total = rg if total is None else {n: tuple(a + b for a, b in zip(total[n], rg[n])) for n in rg}
    views = pack.lora_views(cfg, grad)
    for n in synth.PROJ:
        for k in (0, 1):
            assert normwise_err(views[n][k].cpu().numpy(), total[n][k]) <= TOL, (n, k)


@pytest.mark.parametrize("form", ["d128, a group of 4, bf16 weights, rank 64",
                                  "d128, a group of 3, absmax of 8 bits"])
def test_step(L, form):
    import torch
    from gpu_util import check_stack_grad, workspace
    from layer_streamed_qlora_nf4_b200 import pack
    cfg = dict(CFGS[form], n_layers=2)
    st = Stack(L, cfg, 9)
    T, rows = 140, [[90, 0, 41], [50, 61, 20]]
    prompts = [[30, 0, 0], [0, 61, 9]]
    rng = np.random.default_rng(7)
    tokens = rng.integers(0, cfg["vocab"], (2, T)).astype(np.int32)
    h = st.handle(L, False)
    lora = st.lora.clone()
    grad = torch.full_like(lora, float("nan"))
    loss = L.stream_stack_packed_step(
        h, torch.from_numpy(tokens).cuda(), torch.tensor(rows, dtype=torch.int32, device="cuda"),
        st.emb, st.head, st.gf, lora, grad,
        workspace(L.stream_stack_packed_workspace_bytes(cfg, T, 3)),
        prefix=torch.tensor(prompts, dtype=torch.int32, device="cuda"))
    h.close()
    layers = st.oracle_layers()
    emb, head, gf = (synth.bf16_bits_to_f32(b) for b in (st.emb_bits, st.head_bits, st.gf_bits))
    docs = [op.documents(r, p) for r, p in zip(rows, prompts)]
    ys = [op.targets(tokens[m], docs[m]) for m in (0, 1)]
    n, want, total = sum(int((y >= 0).sum()) for y in ys), 0.0, None
    for m in (0, 1):
        for s, e, pe in docs[m]:
            if e == s:
                continue
            with _Prompt(pe - s):
                lg, c = om.stack_forward(layers, emb, head, gf, tokens[m][None, s:e], cfg)
                _, part, dl = op.cross_entropy(lg.reshape(e - s, -1), ys[m][s:e], None, n)
                want += part
                dh = om.rmsnorm_bwd(dl @ head.astype(np.float64), c["h"], gf, cfg["rms_eps"])
                grads = [None] * len(layers)
                for i in range(len(layers) - 1, -1, -1):
                    dh, grads[i] = om.decoder_layer_bwd(layers[i], c["xs"][i], dh, cfg, e - s)
            total = grads if total is None else [
                {k: tuple(a + b for a, b in zip(t[k], g[k])) for k in g} for t, g in zip(total, grads)]
    assert abs(loss - want) <= 1e-3 * abs(want), (loss, want)
    nf = L.lsq_lora_layout_get(cfg).floats_per_layer
    for i in range(cfg["n_layers"]):
        views = pack.lora_views(cfg, grad[i * nf:(i + 1) * nf])
        for name in synth.PROJ:
            for k in (0, 1):
                check_stack_grad(views[name][k].cpu().numpy(), total[i][name][k], name, (i, k))
    assert L.lsq_device_status(clear=True) == 0


def test_a_head_in_several_chunks(L):
    """A row whose logits are computed in two chunks (more than 4 GiB of logits and their
    gradient) against the same documents as two rows of one chunk each: the loss from the
    row's own logits in fp64, the gradients at the stack's tolerance."""
    import torch
    from gpu_util import check_stack_grad, workspace
    from layer_streamed_qlora_nf4_b200 import pack
    cfg = dict(synth.SMALL, n_layers=1, vocab=synth.QWEN3B["vocab"])
    V, half = cfg["vocab"], 2400
    rows = 2 ** 32 // (6 * V) // 128 * 128
    assert half < rows < 2 * half
    st = Stack(L, cfg, 9, tied=True)
    rng = np.random.default_rng(8)
    tokens = rng.integers(0, V, (1, 2 * half)).astype(np.int32)
    lens = [[1000, 900, 500], [37, 1863, 480]]           # the second half ends in padding
    mask = (rng.random(2 * half) < 0.5).astype(np.uint8)

    def run(n_rows):
        T, docs = 2 * half // n_rows, 6 // n_rows
        h = st.handle(L, True)
        lora = st.lora.clone()
        grad = torch.full_like(lora, float("nan"))
        logits = torch.empty(T, V, device="cuda")
        loss = L.stream_stack_packed_step(
            h, torch.from_numpy(tokens.reshape(n_rows, T)).cuda(),
            torch.tensor(lens, dtype=torch.int32, device="cuda").view(n_rows, docs), st.emb, st.head,
            st.gf, lora, grad, workspace(L.stream_stack_packed_workspace_bytes(cfg, T, docs)),
            loss_mask=torch.from_numpy(mask.reshape(n_rows, T)).cuda(), logits_out=logits)
        h.close()
        return loss, grad.cpu().numpy(), logits
    loss, grad, logits = run(1)
    y = op.targets(tokens[0], op.documents(lens[0] + lens[1]), mask)
    at = np.nonzero(y >= 0)[0]
    want = sum(float(torch.nn.functional.cross_entropy(
        logits[torch.from_numpy(a).cuda()].double(), torch.from_numpy(y[a]).cuda(), reduction="sum"))
        for a in np.array_split(at, 8)) / len(at)
    # sums of 151,936 exponentials, 600 a thread, and of 2400 rows in fp32
    assert abs(loss - want) <= 2.0 ** -13 * want, (loss, want)
    del logits
    loss2, grad2, _ = run(2)
    assert abs(loss - loss2) <= 1e-3 * loss2
    a, b = (pack.lora_views(cfg, torch.from_numpy(g)) for g in (grad, grad2))
    for name in synth.PROJ:
        for k in (0, 1):
            check_stack_grad(a[name][k].numpy(), b[name][k].numpy(), name, k)
    assert L.lsq_device_status(clear=True) == 0
