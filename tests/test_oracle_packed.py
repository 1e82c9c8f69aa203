"""The fp64 oracle of the packed operators and the 8-bit AdamW, pinned by itself:
finite differences, brute-force masks, exhaustive level searches."""
import numpy as np
import pytest

from oracle import packed as op

DOCS = [([5, 0, 1, 7], None, 15), ([4, 6], [2, 6], 10), ([9], [0], 11)]


@pytest.mark.parametrize("lengths,prefix,T", DOCS)
def test_visible_is_the_definition(lengths, prefix, T):
    see = op.visible(T, op.documents(lengths, prefix))
    a = 0
    for k, n in enumerate(lengths):
        p = 0 if prefix is None else prefix[k]
        for i in range(T):
            for j in range(T):
                both = a <= i < a + n and a <= j < a + n
                if both:
                    assert see[i, j] == (j <= i or j < a + p)
                elif a <= i < a + n or a <= j < a + n:
                    assert not see[i, j]
        a += n
    assert not see[a:].any() and not see[:, a:].any()


@pytest.mark.parametrize("lengths,prefix,T", DOCS)
def test_attention_gradient_against_differences(lengths, prefix, T):
    rng = np.random.default_rng(0)
    H, Hkv, d = 4, 2, 3
    docs = op.documents(lengths, prefix)
    x = rng.standard_normal((T, (H + 2 * Hkv) * d))
    w = rng.standard_normal((T, H * d))

    def f(x):
        return float((op.attention_fwd(x, H, Hkv, docs)[0].reshape(T, -1) * w).sum())
    g = op.attention_bwd(x, H, Hkv, docs, w)
    for _ in range(25):
        i, j = rng.integers(T), rng.integers(x.shape[1])
        e = np.zeros_like(x)
        e[i, j] = 1e-5
        # central differences: truncation ~ h^2, rounding ~ 1e-16 / h
        assert abs((f(x + e) - f(x - e)) / 2e-5 - g[i, j]) < 1e-8


def test_cross_entropy_gradient_against_differences():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((4, 9))
    y, w = np.array([3, -1, 0, 8]), np.array([1.0, 5.0, 0.5, 2.0])
    row, loss, g = op.cross_entropy(x, y, w, 3)
    assert row[1] == 0 and not g[1].any()
    assert abs(loss - (w * row).sum() / 3) < 1e-12
    for i in range(4):
        for j in range(9):
            e = np.zeros_like(x)
            e[i, j] = 1e-5
            d = (op.cross_entropy(x + e, y, w, 3)[1] - op.cross_entropy(x - e, y, w, 3)[1]) / 2e-5
            assert abs(d - g[i, j]) < 1e-8


def test_targets_stay_in_the_document_and_out_of_the_prompt():
    docs = op.documents([4, 1, 3], [2, 0, 3])
    assert list(op.targets(np.arange(10, 19), docs)) == [-1, 12, 13, -1, -1, -1, -1, -1, -1]
    mask = np.array([0, 0, 0, 1, 1, 1, 1, 1, 1])
    assert list(op.targets(np.arange(10, 19), docs, mask)) == [-1, -1, 13] + [-1] * 6


@pytest.mark.parametrize("signed", [True, False])
def test_codes_are_the_nearest_root_and_round_trip(signed):
    rng = np.random.default_rng(2)
    x = (rng.standard_normal(700) * np.exp(rng.standard_normal(700) * 2)).astype(np.float32)
    x = x if signed else np.abs(x)
    x[300:310] = 0
    codes, scale = op.encode(x, signed)
    top = 127 if signed else 255
    for b in range(3):
        part = slice(b * 256, (b + 1) * 256)
        a = float(np.abs(x[part]).max())
        assert scale[b] == np.float32(a)
        roots = np.arange(top + 1) / top
        r = (np.abs(x[part].astype(np.float64)) / a) ** (0.5 if signed else 0.25)
        best = np.abs(r[:, None] - roots[None]).argmin(1)
        if not signed:
            best = np.where((x[part] > 0) & (best == 0), 1, best)
        assert np.array_equal(np.abs(codes[part].astype(int)), best)
    assert np.array_equal(op.decode(codes, scale) == 0, codes == 0)
    again, s2 = op.encode(op.decode(codes, scale), signed)
    assert np.array_equal(again, codes) and np.allclose(s2, scale, rtol=1e-6)


def test_adamw_matches_torch():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(3)
    p = rng.standard_normal(50)
    t = torch.nn.Parameter(torch.tensor(p))
    opt = torch.optim.AdamW([t], lr=1e-2, weight_decay=0.1, betas=(0.9, 0.999), eps=1e-8)
    m = v = np.zeros(50, np.float32)
    for step in range(1, 5):
        g = rng.standard_normal(50).astype(np.float32)
        t.grad = torch.tensor(g.astype(np.float64))
        opt.step()
        p, m, v = op.adamw(p, g, m, v, step, 1e-2, 0.1)
    # the fp32 moments and betas: a few 2^-24 of updates of size lr
    assert np.abs(p - t.detach().numpy()).max() < 4 * 1e-2 * 2.0 ** -20


@pytest.mark.parametrize("a,v,code", [(10322846.0, 665658.125, 129),   # 128.5 and 203.5 are the
                                      (8629209.0, 3499999.0, 203)])    # borders next to them
def test_a_code_next_to_a_border_is_chosen_in_whole_numbers(a, v, code):
    """The products that are compared differ by less than a step of fp64."""
    border = int(np.rint(255 * (v / a) ** 0.25 - 0.5))
    diff = int(8 * v) * 510 ** 4 - int(8 * a) * (2 * border + 1) ** 4
    assert abs(diff) < 1000 and code == border + (diff > 0)
    x = np.zeros(256, np.float32)
    x[:2] = a, v
    assert op.encode(x, False)[0][1] == code
