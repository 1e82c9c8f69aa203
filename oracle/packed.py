"""Packed documents and the many-tensor AdamW, plain and slow, in fp64 (numpy).

Attention inside documents: token i of a document [s, e) with a prompt of p tokens
sees the keys [s, max(i + 1, s + p)); the loss of the tokens with a target; the AdamW
update with an 8-bit state.  Test infrastructure only: shares no code with the GPU path.
"""
import numpy as np


def documents(lengths, prefix=None):
    """-> list of (start, end, end of the prompt)."""
    out, a = [], 0
    for k, n in enumerate(lengths):
        p = 0 if prefix is None else int(prefix[k])
        out.append((a, a + int(n), a + p))
        a += int(n)
    return out


def visible(T, docs):
    """Boolean [T, T]: does the row's token see the column's token?"""
    m = np.zeros((T, T), bool)
    for s, e, pe in docs:
        for i in range(s, e):
            m[i, s:max(i + 1, pe)] = True
    return m


def split_heads(qkv, H, Hkv):
    T = qkv.shape[0]
    d = qkv.shape[1] // (H + 2 * Hkv)
    x = np.asarray(qkv, np.float64).reshape(T, H + 2 * Hkv, d)
    return x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]


def attention_fwd(qkv, H, Hkv, docs):
    """-> o [T, H, d], lse [H, T], p [H, T, T]; rows of no document: 0 and -inf."""
    q, k, v = split_heads(qkv, H, Hkv)
    T, _, d = q.shape
    see = visible(T, docs)
    o = np.zeros((T, H, d))
    lse = np.full((H, T), -np.inf)
    p = np.zeros((H, T, T))
    for h in range(H):
        g = h // (H // Hkv)
        for i in range(T):
            at = np.nonzero(see[i])[0]
            if at.size == 0:
                continue
            s = k[at, g] @ q[i, h] / np.sqrt(d)
            top = s.max()
            w = np.exp(s - top)
            lse[h, i] = top + np.log(w.sum())
            p[h, i, at] = w / w.sum()
            o[i, h] = p[h, i, at] @ v[at, g]
    return o, lse, p


def attention_bwd(qkv, H, Hkv, docs, dout):
    """-> dqkv [T, (H + 2 Hkv) d] of sum(o * dout)."""
    q, k, v = split_heads(qkv, H, Hkv)
    T, _, d = q.shape
    o, _, p = attention_fwd(qkv, H, Hkv, docs)
    do = np.asarray(dout, np.float64).reshape(T, H, d)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for h in range(H):
        g = h // (H // Hkv)
        dp = do[:, h] @ v[:, g].T
        delta = (do[:, h] * o[:, h]).sum(1)
        ds = p[h] * (dp - delta[:, None]) / np.sqrt(d)
        dq[:, h] = ds @ k[:, g]
        dk[:, g] += ds.T @ q[:, h]
        dv[:, g] += p[h].T @ do[:, h]
    return np.concatenate([dq, dk, dv], 1).reshape(T, -1)


def targets(tokens, docs, loss_mask=None):
    T = len(tokens)
    y = np.full(T, -1, np.int64)
    for s, e, pe in docs:
        for t in range(s, e - 1):
            if t + 1 >= pe and tokens[t + 1] >= 0 and (loss_mask is None or loss_mask[t + 1]):
                y[t] = tokens[t + 1]
    return y


def cross_entropy(logits, y, weight=None, count=None):
    """-> row losses, loss, dlogits."""
    x = np.asarray(logits, np.float64)
    T, V = x.shape
    row, grad, loss = np.zeros(T), np.zeros((T, V)), 0.0
    for t in range(T):
        if not 0 <= y[t] < V:
            continue
        c = (1.0 if weight is None else float(weight[t])) / (1.0 if count is None else max(1, count))
        top = x[t].max()
        lse = top + np.log(np.exp(x[t] - top).sum())
        row[t] = lse - x[t, y[t]]
        loss += c * row[t]
        grad[t] = c * np.exp(x[t] - lse)
        grad[t, y[t]] -= c
    return row, loss, grad


BLOCK = 256
TINY = float(np.finfo(np.float32).tiny)


def decode(codes, scale):
    """8-bit codes (int8: m, uint8: v) to fp32 values: scale * fl32(level)."""
    c = codes.astype(np.float64)
    level = c * np.abs(c) / 127.0 ** 2 if codes.dtype == np.int8 else c ** 4 / 255.0 ** 4
    a = np.repeat(np.asarray(scale, np.float32), BLOCK)[:len(c)]
    return a * level.astype(np.float32)


def _above(v, a, c, top, power):
    """Is v / a above, at or below the border ((2 c + 1) / (2 top))^power?  1, 0 or -1, in
    whole numbers: an fp32 number is a whole number of 2^-149."""
    l = int(v * 2.0 ** 149) * (2 * top) ** power
    r = int(a * 2.0 ** 149) * (2 * c + 1) ** power
    return (l > r) - (l < r)


def encode(x, signed):
    """fp32 values to (codes, scale): the nearest root (a tie: the even one).  Next to a border
    between two codes the choice is made in whole numbers."""
    x = np.asarray(x, np.float32)
    n = len(x)
    scale = np.zeros((n + BLOCK - 1) // BLOCK, np.float32)
    codes = np.zeros(n, np.int8 if signed else np.uint8)
    top, power = (127, 2) if signed else (255, 4)
    for b in range(len(scale)):
        v = x[b * BLOCK:(b + 1) * BLOCK].astype(np.float64)
        a = np.abs(v).max()
        if a < TINY:
            continue
        scale[b] = a
        r = top * (np.abs(v) / a) ** (1.0 / power)
        c = np.minimum(np.rint(r), top)
        low = np.floor(r)
        for i in np.nonzero(np.abs(r - low - 0.5) < 1e-9)[0]:
            k = int(low[i])
            c[i] = k + (1, k & 1, 0)[1 - _above(abs(v[i]), a, k, top, power)]
        if signed:
            c = np.sign(v) * c
        else:
            c = np.where((v > 0) & (c < 1), 1, c)
        codes[b * BLOCK:(b + 1) * BLOCK] = c
    return codes, scale


def adamw(p, g, m, v, step, lr, wd, b1=0.9, b2=0.999, eps=1e-8):
    """One update of one tensor: p in fp64; the moments in fp32, every product and sum
    rounded once.  m, v: fp32 arrays."""
    f = np.float32
    b1, b2, g = f(b1), f(b2), np.asarray(g, f)
    m1 = b1 * m.astype(f) + f(1.0 - float(b1)) * g
    v1 = b2 * v.astype(f) + (f(1.0 - float(b2)) * g) * g
    mh = m1.astype(np.float64) / (1.0 - float(b1) ** step)
    vh = v1.astype(np.float64) / (1.0 - float(b2) ** step)
    p = np.asarray(p, np.float64)
    lr, wd = float(f(lr)), float(f(wd))
    return p * (1.0 - lr * wd) - lr * mh / (np.sqrt(vh) + float(f(eps))), m1, v1
