"""The operators of a packed fine-tuning step, and the cases they are timed on.

A packed step puts several documents of different lengths behind one another in one
row of tokens.  Its operators: attention that stays inside each document (forward, and
forward with backward), the cross-entropy over the vocabulary with its gradient, for
the tokens that are trained on, and AdamW over many tensors at once, with its state in
8 or in 32 bits.

``own`` false: their plain form in elementary torch operations, in fp32, rounded once
at the end.  ``own`` true: the library's entry points, called as a training program
calls them.  ``exact``: the same results from the definitions in fp64, written apart.
"""
import math
import random

import torch

own = False

BLOCK = 256            # state elements per scale of the 8-bit AdamW
# One decoder layer's LoRA factors of the 8B-shaped stack (rank 16): A and B of q, k, v,
# o, gate, up and down.
LORA_8B = "65536,65536,65536,16384,65536,16384,65536,65536,65536,229376,65536,229376,229376,65536"


# ------------------------------------------------------------------ the cases
def listed():
    attn8b = dict(heads=32, kv_heads=8, dim=128)
    attn3b = dict(heads=16, kv_heads=2, dim=128)
    return [
        # one micro-batch of the 8B-shaped stack: 512 tokens, five short documents
        dict(name="attn_fwd_512", op="attn_fwd", T=512, docs="201,7,118,96,90", prefix=False, **attn8b),
        # the 3B-shaped stack's batch (8 x 2048 tokens) as packed chats, each with a prompt that
        # is read in both directions; the last row's tail is padding
        dict(name="attn_fwd_16384_prefix", op="attn_fwd", T=16384, docs="32..2048", doc_seed=3, pad=200, prefix=True, **attn3b),
        # one long document at the 8B shapes: the largest call
        dict(name="attn_fwd_16384_long", op="attn_fwd", T=16384, docs="16384", prefix=False, **attn8b),
        # a layer's recomputing backward on the 8B micro-batch
        dict(name="attn_train_512", op="attn_train", T=512, docs="201,7,118,96,90", prefix=False, **attn8b),
        # the same on the 3B-shaped batch
        dict(name="attn_train_16384", op="attn_train", T=16384, docs="32..2048", doc_seed=4, pad=77, prefix=False, **attn3b),
        # the smallest call: a small 64-wide model on a few short documents, one token and none
        # among them, where latency counts
        dict(name="attn_train_167", op="attn_train", T=167, docs="80,1,0,79", pad=7, prefix=True, heads=8, kv_heads=2, dim=64),
        # the 8B vocabulary, one micro-batch, most tokens trained on
        dict(name="loss_512x128256", op="loss", T=512, V=128256, trained=0.9),
        # the 3B vocabulary, one chunk of the head, answers only (long prompts)
        dict(name="loss_2048x151936", op="loss", T=2048, V=151936, trained=0.4),
        # a small model's few tokens, odd vocabulary: latency
        dict(name="loss_7x1001", op="loss", T=7, V=1001, trained=0.8),
        # the LoRA factors of the whole 8B-shaped stack, state in 8 bits
        dict(name="adamw8_448", op="adamw", sizes=LORA_8B, repeat=32, bits=8, grad="fp32"),
        # the same with the state in 32 bits
        dict(name="adamw32_448", op="adamw", sizes=LORA_8B, repeat=32, bits=32, grad="fp32"),
        # a few ragged tensors with bf16 gradients: norms, biases and a small factor
        dict(name="adamw8_ragged", op="adamw", sizes="8192,17,512,1,1408,255,257,5000", repeat=3, bits=8, grad="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("attn_fwd", "attn_train", "loss", "adamw"))
    if op in ("attn_fwd", "attn_train"):
        # a backward of the longest documents would cost more than the largest listed case
        T = _log(rng, 1, 16384 if op == "attn_fwd" else 8192)
        heads, kv = rng.choice(((32, 8), (16, 2), (8, 2), (6, 2), (4, 4), (5, 1)))
        hi = _log(rng, max(1, T // 32), T)
        lo = _log(rng, max(1, hi // 16), hi)
        return dict(op=op, T=T, docs="%d..%d" % (lo, hi), doc_seed=rng.randrange(1 << 30),
                    pad=rng.randrange(0, T // 4 + 1), prefix=rng.random() < 0.4, heads=heads,
                    kv_heads=kv, dim=rng.choice((64, 128, 128)))
    if op == "loss":
        V = _log(rng, 2, 262144)
        V += (-V) % 8 if rng.random() < 0.5 else 0
        return dict(op=op, T=_log(rng, 1, max(1, min(4096, 2048 * 151936 // V))), V=V,
                    trained=rng.choice((0.0, 0.3, 0.7, 1.0)))
    n = _log(rng, 1, 600)
    top = max(2, min(4000000, 40000000 // n))
    sizes = ",".join(str(_log(rng, 1, top)) for _ in range(n))
    return dict(op=op, sizes=sizes, repeat=1, bits=rng.choice((8, 8, 32)), grad=rng.choice(("fp32", "bf16")))


def _documents(case):
    """Lengths of the documents, and of the prompt of each that is read in both directions."""
    if ".." in case["docs"]:
        lo, hi = (int(x) for x in case["docs"].split(".."))
        rng = random.Random(case["doc_seed"])
        room, lens = case["T"] - case.get("pad", 0), []
        while room > 0 and len(lens) < 4096:
            lens.append(min(room, _log(rng, lo, hi)))
            room -= lens[-1]
    else:
        lens = [int(x) for x in case["docs"].split(",")]
    rng = random.Random(len(lens))
    return lens, [rng.randint(0, n) if case["prefix"] else 0 for n in lens]


def _sizes(case):
    return [int(x) for x in case["sizes"].split(",")] * case["repeat"]


def work(case):
    if case["op"] == "loss":
        rows = round(case["T"] * case["trained"])
        return {"bytes": case["V"] * (4 * rows + 2 * case["T"]) + 8 * case["T"], "flops": 4 * case["V"] * rows}
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        g = 4 if case["grad"] == "fp32" else 2
        # 8 bits: the codes and scales read and written, and the values they stand for written
        state = 16 if case["bits"] == 32 else 4 + 4 * 4 / BLOCK + 8
        return {"bytes": n * (8 + g + state), "flops": 20 * n}
    T, H, d = case["T"], case["heads"], case["dim"]
    # token i sees the document up to itself, and all of its prompt
    pairs = sum(n * (n + 1) // 2 + p * (p - 1) // 2 for n, p in zip(*_documents(case)))
    size = 2 * T * (H + 2 * case["kv_heads"]) * d + 2 * T * H * d + 4 * T * H
    if case["op"] == "attn_fwd":
        return {"bytes": size, "flops": 4 * H * d * pairs}
    size += 2 * T * H * d + 2 * T * (H + 2 * case["kv_heads"]) * d
    return {"bytes": size, "flops": 14 * H * d * pairs}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=case)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    if case["op"] in ("attn_fwd", "attn_train"):
        T, H, kv, d = case["T"], case["heads"], case["kv_heads"], case["dim"]
        s["lens"], s["prompts"] = _documents(case)
        s["lengths"] = torch.tensor(s["lens"], dtype=torch.int32, device="cuda")
        s["prefix"] = torch.tensor(s["prompts"], dtype=torch.int32, device="cuda") if case["prefix"] else None
        s["qkv"] = normal(T, (H + 2 * kv) * d).half()
        s["o"] = torch.empty(T, H * d, dtype=torch.float16, device="cuda")
        s["lse"] = torch.empty(H, T, device="cuda")
        if own:
            from layer_streamed_qlora_nf4_b200 import lib
            s["index"] = lib.PackedIndex(T, len(s["lens"]))
        if case["op"] == "attn_train":
            # gradients of a mean loss: small, and of different size from token to token
            s["dout"] = (normal(T, H * d) * torch.exp(normal(T, 1)) * 1e-5).bfloat16()
            s["dqkv"] = torch.empty(T, (H + 2 * kv) * d, dtype=torch.bfloat16, device="cuda")
            if own:
                s["ws"] = torch.empty(lib.packed_attention_workspace_bytes(T, H, kv, d), dtype=torch.uint8, device="cuda")
    elif case["op"] == "loss":
        T, V = case["T"], case["V"]
        s["logits"] = normal(T, V) * 2.5
        targets = torch.randint(0, V, (T,), device="cuda", generator=g, dtype=torch.int32)
        skip = torch.rand(T, device="cuda", generator=g).argsort() >= round(T * case["trained"])
        s["targets"] = torch.where(skip, -1, targets).int()
        s["count"] = (s["targets"] >= 0).sum(dtype=torch.int32).reshape(1)
        s["dlogits"] = torch.empty(T, V, dtype=torch.bfloat16, device="cuda")
        s["row_loss"] = torch.empty(T, device="cuda")
        s["loss"] = torch.empty(1, device="cuda")
    else:
        # every tensor lies at a multiple of 256 elements of one buffer, as its state does
        sizes = _sizes(case)
        spans = [-(-n // BLOCK) * BLOCK for n in sizes]
        total = sum(spans)
        s["sizes"], s["starts"] = sizes, [0]
        for n in spans[:-1]:
            s["starts"].append(s["starts"][-1] + n)
        n_of, span_of = (torch.tensor(x, device="cuda") for x in (sizes, spans))
        live = torch.arange(total, device="cuda") - torch.repeat_interleave(torch.tensor(s["starts"], device="cuda"), span_of)
        live = (live < torch.repeat_interleave(n_of, span_of)).float()
        scale = torch.repeat_interleave(torch.exp(normal(len(sizes))) * 1e-4, span_of) * live
        s["p"] = normal(total) * 0.02 * live
        s["g"] = normal(total) * scale
        s["g"] = s["g"].bfloat16() if case["grad"] == "bf16" else s["g"]
        m, v = normal(total) * scale * 0.3, (0.2 + normal(total) ** 2) * scale * scale
        # the A factors learn at 2e-4 with decay, the B factors at twice that without
        s["lr"] = [2e-4, 4e-4] * (len(sizes) // 2 + 1)
        s["wd"] = [0.01, 0.0] * (len(sizes) // 2 + 1)
        blocks = span_of // BLOCK
        s["lr_b"], s["wd_b"] = (torch.repeat_interleave(torch.tensor(x[:len(sizes)], device="cuda"), blocks)[:, None]
                                for x in (s["lr"], s["wd"]))
        s["step"] = 10
        if case["bits"] == 8:
            (s["m"], s["ms"]), (s["v"], s["vs"]) = _encode_m(m.view(-1, BLOCK)), _encode_v(v.view(-1, BLOCK))
            s["m"], s["v"] = s["m"].reshape(-1), s["v"].reshape(-1)
            s["m_out"], s["v_out"] = torch.empty(total, device="cuda"), torch.empty(total, device="cuda")
        else:
            s["m"], s["v"], s["ms"], s["vs"] = m, v, None, None
        if own:
            from layer_streamed_qlora_nf4_b200 import lib

            def parts(t, unit=1):
                return None if t is None else [t[a // unit:a // unit + -(-n // unit)] for a, n in zip(s["starts"], sizes)]
            s["opt"] = lib.AdamWMulti(parts(s["p"]), parts(s["g"]), parts(s["m"]), parts(s["v"]), lr=s["lr"][:len(sizes)],
                                      weight_decay=s["wd"][:len(sizes)], m_scale=parts(s["ms"], BLOCK), v_scale=parts(s["vs"], BLOCK))
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        from layer_streamed_qlora_nf4_b200 import lib
        if op in ("attn_fwd", "attn_train"):
            H, kv = s["case"]["heads"], s["case"]["kv_heads"]
            lib.packed_index(s["lengths"], s["index"], prefix=s["prefix"])
            lib.packed_attention_fwd(s["qkv"], s["index"], H, kv, s["o"], s["lse"])
            if op == "attn_fwd":
                return s["o"], s["lse"]
            lib.packed_attention_bwd(s["qkv"], s["index"], s["o"], s["lse"], s["dout"], H, kv, s["dqkv"], s["ws"])
            return s["o"], s["lse"], s["dqkv"]
        if op == "loss":
            lib.packed_cross_entropy(s["logits"], s["targets"], s["row_loss"], s["loss"], dlogits=s["dlogits"], count=s["count"])
            return s["row_loss"], s["loss"], s["dlogits"]
        s["opt"].step(s["step"])
        if s["case"]["bits"] == 32:
            return s["p"], s["m"], s["v"]
        lib.adamw_state_dequantize(s["m"], s["ms"], s["m_out"])
        lib.adamw_state_dequantize(s["v"], s["vs"], s["v_out"])
        return s["p"], s["m_out"], s["v_out"]
    return {"attn_fwd": _plain_attention, "attn_train": _plain_attention, "loss": _plain_loss, "adamw": _plain_adamw}[op](s)


# ------------------------------------------------------------------ the plain forms
def _plain_attention(s):
    c = s["case"]
    T, H, kv, d = c["T"], c["heads"], c["kv_heads"], c["dim"]
    G, scale = H // kv, 1.0 / math.sqrt(d)
    o = torch.zeros(T, kv, G, d, device="cuda")
    lse = torch.full((kv, G, T), -math.inf, device="cuda")
    x = s["qkv"].float()
    q, k, v = x[:, :H * d].view(T, kv, G, d), x[:, H * d:(H + kv) * d].view(T, kv, d), x[:, (H + kv) * d:].view(T, kv, d)
    train = c["op"] == "attn_train"
    if train:
        do = s["dout"].float().view(T, kv, G, d)
        grad = torch.zeros_like(x)
        dq, dk, dv = grad[:, :H * d].view(T, kv, G, d), grad[:, H * d:(H + kv) * d].view(T, kv, d), grad[:, (H + kv) * d:].view(T, kv, d)
    a = 0
    for n, prompt in zip(s["lens"], s["prompts"]):
        if n == 0:
            continue
        e, at = a + n, torch.arange(n, device="cuda")
        seen = (at[None, :] <= at[:, None]) | (at[None, :] < prompt)
        heads = max(1, min(kv, (1 << 30) // (n * n * G)))  # kv heads at a time
        for h in range(0, kv, heads):
            hs = slice(h, min(kv, h + heads))
            qh, kh, vh = q[a:e, hs].permute(1, 2, 0, 3), k[a:e, hs].permute(1, 0, 2)[:, None], v[a:e, hs].permute(1, 0, 2)[:, None]
            p = (qh @ kh.transpose(-1, -2)).mul_(scale).masked_fill_(~seen, -math.inf)
            top = p.amax(-1, keepdim=True)
            p = p.sub_(top).exp_()
            z = p.sum(-1, keepdim=True)
            p = p.div_(z)
            oh = p @ vh
            o[a:e, hs] = oh.permute(2, 0, 1, 3)
            lse[hs, :, a:e] = (top + z.log())[..., 0]
            if train:
                doh = do[a:e, hs].permute(1, 2, 0, 3)
                dv[a:e, hs] = (p.transpose(-1, -2) @ doh).sum(1).permute(1, 0, 2)
                ds = (doh @ vh.transpose(-1, -2)).sub_((doh * oh).sum(-1, keepdim=True)).mul_(p).mul_(scale)
                dq[a:e, hs] = (ds @ kh).permute(2, 0, 1, 3)
                dk[a:e, hs] = (ds.transpose(-1, -2) @ qh).sum(1).permute(1, 0, 2)
        a = e
    out = o.reshape(T, H * d).half(), lse.reshape(H, T)
    return (*out, grad.bfloat16()) if train else out


def _plain_loss(s):
    logits, y = s["logits"], s["targets"].long()
    on = y >= 0
    part = on.float() / s["count"].clamp(min=1)
    top = logits.amax(-1, keepdim=True)
    e = (logits - top).exp()
    z = e.sum(-1, keepdim=True)
    row = torch.where(on, top[:, 0] + z[:, 0].log() - logits.gather(1, y.clamp(min=0)[:, None])[:, 0], 0.0)
    e = e.div_(z)
    e.scatter_add_(1, y.clamp(min=0)[:, None], torch.full_like(z, -1.0))
    return row, (row * part).sum().reshape(1), e.mul_(part[:, None]).bfloat16()


# The 8-bit state, blocks of 256 with the block's largest magnitude as their scale.  m: a sign and
# 127 levels, level c at (c / 127)^2; v: 255 levels, level c at (c / 255)^4, and none but an exact
# zero is stored as zero.  The running state is an fp32 number (each product and sum of its update
# rounded), and its code that of the nearest root: a choice next to a border, so made in fp64.
def _scale(top):
    return torch.where(top < torch.finfo(torch.float32).tiny, torch.zeros_like(top), top)


def _encode_m(m):
    a = _scale(m.abs().amax(1))
    x = m.double().abs() / torch.where(a > 0, a, math.inf).double()[:, None]
    return (m.sign() * (127.0 * x.sqrt()).round()).to(torch.int8), a


def _encode_v(v):
    a = _scale(v.amax(1))
    q = (255.0 * (v.double() / torch.where(a > 0, a, math.inf).double()[:, None]).sqrt().sqrt()).round()
    return torch.where((v > 0) & (a > 0)[:, None], q.clamp(min=1.0), q).to(torch.uint8), a


def _decode_m(c, a):
    c = c.double()
    return a[:, None] * (c * c.abs() / 127.0 ** 2).float()


def _decode_v(c, a):
    return a[:, None] * (c.double() ** 4 / 255.0 ** 4).float()


def _f32(x):
    return torch.tensor(x, dtype=torch.float32).item()


def _plain_adamw(s):
    b1, b2, eps = _f32(0.9), _f32(0.999), 1e-8
    bits8 = s["case"]["bits"] == 8
    p, g = s["p"].view(-1, BLOCK), s["g"].view(-1, BLOCK).float()
    m, v = s["m"].view(-1, BLOCK), s["v"].view(-1, BLOCK)
    if bits8:
        m, v = _decode_m(m, s["ms"]), _decode_v(v, s["vs"])
    m = b1 * m + (1 - b1) * g
    v = b2 * v + ((1 - b2) * g) * g
    mh, vh = m / (1 - b1 ** s["step"]), v / (1 - b2 ** s["step"])
    p.copy_(p * (1 - s["lr_b"] * s["wd_b"]) - s["lr_b"] * mh / (vh.sqrt() + eps))
    if bits8:
        (mc, s["ms"]), (vc, s["vs"]) = _encode_m(m), _encode_v(v)
        m, v = _decode_m(mc, s["ms"]), _decode_v(vc, s["vs"])
        s["m"], s["v"] = mc.view(-1), vc.view(-1)
    else:
        s["m"], s["v"] = m.view(-1), v.view(-1)
    return s["p"], m.reshape(-1), v.reshape(-1)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("attn_fwd", "attn_train"):
        return _exact_attention(s)
    if case["op"] == "loss":
        x, y = s["logits"].double(), s["targets"].long()
        n = max(1, int((y >= 0).sum()))
        row = torch.zeros(case["T"], dtype=torch.float64, device="cuda")
        grad = torch.zeros_like(x)
        at = (y >= 0).nonzero()[:, 0]
        if at.numel():
            log_p = x[at] - torch.logsumexp(x[at], 1)[:, None]
            row[at] = -log_p[torch.arange(at.numel(), device="cuda"), y[at]]
            grad[at] = (log_p.exp() - torch.nn.functional.one_hot(y[at], case["V"])) / n
        return row, row.sum().reshape(1) / n, grad
    p, g = s["p"].double(), s["g"].double()
    b1, b2, t = _f32(0.9), _f32(0.999), s["step"]

    def per(x):
        return torch.repeat_interleave(x.double(), BLOCK)

    def r(x):  # to an fp32 number and back
        return x.float().double()
    m, v = s["m"].double(), s["v"].double()
    if case["bits"] == 8:  # levels, products and sums are fp32 numbers
        m, v = r(per(s["ms"]) * r(m.sign() * (m / 127) ** 2)), r(per(s["vs"]) * r((v / 255) ** 4))
        m, v = r(r(b1 * m) + r(_f32(1 - b1) * g)), r(r(b2 * v) + r(r(_f32(1 - b2) * g) * g))
    else:
        m, v = m + (1 - b1) * (g - m), v + (1 - b2) * (g ** 2 - v)
    lr, wd = per(s["lr_b"][:, 0]), per(s["wd_b"][:, 0])
    p = p - lr * (wd * p + (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)) ** 0.5 + 1e-8))
    if case["bits"] == 8:
        a = per(m.view(-1, BLOCK).abs().amax(1))
        c = torch.round(127 * (m.abs() / a.clamp(min=1e-300)) ** 0.5)
        m = a * m.sign() * (c / 127) ** 2
        a = per(v.view(-1, BLOCK).amax(1))
        c = torch.round(255 * (v / a.clamp(min=1e-300)) ** 0.25)
        c = torch.where((v > 0) & (c < 1), 1.0, c)
        v = a * (c / 255) ** 4
    return p, m, v


def _exact_attention(s):
    c = s["case"]
    T, H, kv, d = c["T"], c["heads"], c["kv_heads"], c["dim"]
    train = c["op"] == "attn_train"
    x = s["qkv"].double().requires_grad_(train)
    rows = x.view(T, H + 2 * kv, d)
    o = torch.zeros(T, H, d, dtype=torch.float64, device="cuda")
    lse = torch.full((H, T), -math.inf, dtype=torch.float64, device="cuda")
    start = 0
    grad = torch.zeros_like(x)
    for n, prompt in zip(s["lens"], s["prompts"]):
        here = torch.arange(start, start + n, device="cuda")
        for h in range(H) if n else ():
            q, k, v = rows[here, h], rows[here, H + h // (H // kv)], rows[here, H + kv + h // (H // kv)]
            last = torch.maximum(here, torch.full_like(here, start + prompt - 1))
            score = torch.where(here[None, :] > last[:, None], -math.inf, q @ k.T / d ** 0.5)
            lse[h, here] = torch.logsumexp(score, 1).detach()
            out = torch.softmax(score, 1) @ v
            o[here, h] = out.detach()
            if train:
                grad += torch.autograd.grad(out, x, s["dout"].double().view(T, H, d)[here, h])[0]
        start += n
    return (o.view(T, H * d), lse, grad) if train else (o.view(T, H * d), lse)
