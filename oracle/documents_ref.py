"""The operators of a training step over packed documents in 64 bits: head norms with rotary positions, the softmax
cross entropy of hidden states, AdamW over many tensors with 8-bit moments. Plain torch on float64 tensors of any
device, from the definitions; pinned by tests/test_documents_pins.py. Beside each result stand the bounds of what a
kernel may be off, from the roundings that its definition allows: U = 2^-24 for each fp32 operation, half a step of the
output's type for each stored value."""
import math

import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


# ---------------------------------------------------------------- norms and rotation

def turns(rot, base=10000.0, scaling="plain", factor=1.0, context=1024, fast=32.0, slow=1.0):
    """Fractions of a turn per position, as Python floats."""
    if scaling == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    out = []
    for j in range(rot // 2):
        f = math.exp(-2 * j / rot * math.log(base)) / (2 * math.pi)
        if scaling == "linear":
            f = f / factor
        if scaling == "parts":
            n = f * context  # turns over the model's own context
            w = 0.0 if n < slow else 1.0 if n > fast else (n - slow) / (fast - slow)
            f = w * f + (1 - w) * f / factor
        out.append(f)
    return out


def _pairs(rot, interleaved):
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def _cos_sin(pos, turn):
    """cos and sin of pos * turn turns [rows, 1, rot / 2]; turn in units of 2^-64 (int64), reduced exactly."""
    p, t = pos.to(torch.int64)[:, None], turn.to(torch.int64)[None]
    # the product modulo 2^64, as a signed fraction of a turn: int64 products wrap
    a = (p * t).double() * 2.0 ** -64
    return torch.cos(2 * math.pi * a)[:, None], torch.sin(2 * math.pi * a)[:, None]


def rotary(x, pos, turn, gamma=None, eps=None, interleaved=False, amplitude=1.0):
    """y of x [rows, heads, hd] (float64), and the bound of its fp32 arithmetic."""
    hd, rot = x.shape[-1], 2 * turn.shape[0]
    n = x
    if eps is not None:
        n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        if gamma is not None:
            n = n * gamma
    cos, sin = _cos_sin(pos, turn)
    a, b = (i.to(x.device) for i in _pairs(rot, interleaved))
    y, size = n.clone(), n.abs()
    y[..., a] = amplitude * (n[..., a] * cos - n[..., b] * sin)
    y[..., b] = amplitude * (n[..., a] * sin + n[..., b] * cos)
    both = abs(amplitude) * (n[..., a].abs() + n[..., b].abs())
    size[..., a] = both
    size[..., b] = both
    # the norm: hd products and sums, a root and three products; cos and sin: the angle's 2^-25 of half a turn and
    # two units of sincospi; the rotation: three operations
    return y, size * U * ((hd + 8 if eps is not None else 0) + 16)


def rotary_backward(dy, x, pos, turn, gamma=None, eps=None, interleaved=False, amplitude=1.0):
    """dx, dgamma (or None) and their bounds."""
    hd, rot = dy.shape[-1], 2 * turn.shape[0]
    cos, sin = _cos_sin(pos, turn)
    a, b = (i.to(dy.device) for i in _pairs(rot, interleaved))
    dn, size = dy.clone(), dy.abs()
    dn[..., a] = amplitude * (dy[..., a] * cos + dy[..., b] * sin)
    dn[..., b] = amplitude * (dy[..., b] * cos - dy[..., a] * sin)
    both = abs(amplitude) * (dy[..., a].abs() + dy[..., b].abs())
    size[..., a] = both
    size[..., b] = both
    if eps is None:
        return dn, None, size * U * 16, None
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    xhat = x * r
    g = torch.ones_like(x[0, 0]) if gamma is None else gamma
    d = dn * g
    dx = r * (d - xhat * (d * xhat).mean(-1, keepdim=True))
    grown = size * g.abs()
    bound = r * (grown + xhat.abs() * (grown * xhat.abs()).mean(-1, keepdim=True)) * U * (2 * hd + 40)
    terms = (size * xhat.abs()).sum((0, 1))
    # a sum in any order is off by at most its length in units of its terms' sizes
    return dx, (dn * xhat).sum((0, 1)), bound, terms * U * (hd + 40 + dy.shape[0] * dy.shape[1])


# ---------------------------------------------------------------- cross entropy of hidden states

def classifier(x, w, targets, V):
    """losses, lse [N], and their bounds (fp32 sums of exact products on the tensor cores, or fp32 products)."""
    w = w[:V]
    t = torch.where((targets < 0) | (targets >= V), 0, targets).long()
    z = x @ w.T
    lse = torch.logsumexp(z, 1)
    zt = z.gather(1, t[:, None])[:, 0]
    losses = lse - zt
    # each logit: C products summed in fp32 (the accumulators may drop a bit more than a rounding: 2 U a term)
    off = 2 * (x.shape[1] + 4) * U * (x.abs() @ w.abs().T)
    p = torch.exp(z - lse[:, None])
    # the weighted error of the logits reaches lse; exponentials to 8 U, V sums in parts of at most 160 + V / 128
    soft = (p * off).sum(1) + (24 + 160 + V / 128) * U
    top = z.amax(1)
    return losses, lse, soft + off.gather(1, t[:, None])[:, 0] + 8 * U * (losses + (top - zt)), \
        soft + 4 * U * (lse.abs() + top.abs())


def classifier_backward(x, w, targets, V, dloss, dlse, dtype):
    """dx [N, C], dw [V, C] and the bounds of what kernels of this type (dz stored in it) may be off, without the
    rounding of the outputs themselves. w [>= V, C]; the rows of no weight (dloss = dlse = 0) have dz = 0."""
    w = w[:V]
    n = x.shape[0]
    zero = torch.zeros(n, dtype=torch.float64, device=x.device)
    d = zero if dloss is None else dloss
    a = d + (zero if dlse is None else dlse)
    t = torch.where((targets < 0) | (targets >= V), 0, targets).long()
    z = x @ w.T
    lse = torch.logsumexp(z, 1, keepdim=True)
    p = torch.exp(z - lse)
    dz = p * a[:, None]
    dz[torch.arange(n, device=x.device), t] -= d
    counts = (a != 0) | (d != 0)
    dz[~counts] = 0
    p[~counts] = 0
    off = 2 * (x.shape[1] + 4) * U * (x.abs() @ w.abs().T)
    # p: its logit's error, lse's rounding and error (its own bound, above), the exponential
    far = off + (p * off).sum(1, keepdim=True) + U * (6 * lse.abs() + 2 * z.abs() + 200 + V / 128)
    edz = a.abs()[:, None] * p * far + U * 4 * (dz.abs() + d.abs()[:, None] * (p > 0))
    edz = edz + HALF[dtype] * (dz.abs() + edz)
    size = dz.abs() + edz
    # sums of V (or N) products in fp32, 2 U a term, and the pieces' sums
    return dz @ w, dz.T @ x, edz @ w.abs() + 2 * (V + 64) * U * (size @ w.abs()), \
        edz.T @ x.abs() + 2 * (n + 64) * U * (size.T @ x.abs())


# ---------------------------------------------------------------- AdamW with 8-bit moments

GOLDEN = 0x9E3779B97F4A7C15


def _wrap(z):
    return z - (1 << 64) if z >> 63 else z


def mix(z):
    """splitmix64's finaliser on int64 tensors (or Python integers)."""
    if isinstance(z, int):
        z &= (1 << 64) - 1
        z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9 & (1 << 64) - 1
        z = (z ^ (z >> 27)) * 0x94D049BB133111EB & (1 << 64) - 1
        return z ^ (z >> 31)
    z = (z ^ ((z >> 30) & ((1 << 34) - 1))) * _wrap(0xBF58476D1CE4E5B9)
    z = (z ^ ((z >> 27) & ((1 << 37) - 1))) * _wrap(0x94D049BB133111EB)
    return z ^ ((z >> 31) & ((1 << 33) - 1))


def draws(n, tensor, t, seed, device="cpu", start=0):
    """u of the first and of the second moment's rounding for n values of a tensor, from the start-th (even) on."""
    key = mix((seed + t * GOLDEN) & ((1 << 64) - 1))
    pair = torch.arange((n + 1) // 2, dtype=torch.int64, device=device) + start // 2
    r = mix(((tensor << 40) + pair) * _wrap(GOLDEN) + _wrap(key))
    part = lambda i: ((r >> i) & 0xFFFF).double() / 65536  # noqa: E731
    return torch.stack((part(0), part(32)), 1).flatten()[:n], torch.stack((part(16), part(48)), 1).flatten()[:n]


KINDS = {"m": (7, 7, True), "v": (15, 14, False)}  # exponent bias, exponent of a block's largest value, sign


def values(code, scale, kind):
    """What codes (uint8 [n]) under their blocks' scales (uint8 [ceil(n / 128)]) stand for, float64."""
    bias, _, signed = KINDS[kind]
    c = code.long()
    k = c & 127 if signed else c
    nan = k == (127 if signed else 255)
    e, f = k >> 3, (k & 7).double()
    y = torch.where(e > 0, (8 + f) * torch.exp2((e - bias - 3).double()), f * 2.0 ** (-2 - bias))
    y = torch.where(nan, math.nan, y) * torch.exp2(scale.long().clamp(1, 254)[torch.arange(len(c), device=c.device) // 128]
                                                   .double() - 127)
    return torch.where(c >= 128, -y, y) if signed else y


def scales(x, kind):
    """The scale bytes of the finite values of x [n]."""
    _, top, _ = KINDS[kind]
    n = len(x)
    size = torch.zeros(-(-n // 128) * 128, dtype=torch.float64, device=x.device)
    size[:n] = torch.where(torch.isfinite(x), x.abs(), 0.0)
    largest = size.view(-1, 128).amax(1)
    e = torch.floor(torch.log2(largest.clamp_min(2.0 ** -130)))
    return (e - top + 127).clamp(1, 254).long()


def stored(x, scale, u, kind, off=0.0):
    """The value that x [n] is stored as under these scale bytes, rounded with u shifted by `off` codes (0: as
    defined; a small shift either way brackets what rounding errors of x may do)."""
    bias, _, signed = KINDS[kind]
    unit = torch.exp2(scale[torch.arange(len(x), device=x.device) // 128].double() - 127)
    y = x.abs() / unit
    e = torch.floor(torch.log2(y.clamp_min(2.0 ** -60))).clamp_min(1 - bias)
    step = torch.exp2(e - 3)
    q = torch.floor(y / step + u + off).clamp_min(0) * step
    if not signed:
        q = torch.where((x > 0) & (q == 0), 2.0 ** (-2 - bias), q)
    q = torch.where(torch.isfinite(x), q, math.nan)
    return torch.sign(x) * q * unit


def adamw(theta, g, m, v, lr, b1, b2, eps, wd, t, factor):
    """theta, m, v after a step (float64), lr .. eps as the fp32 values that they are passed as."""
    lr, b1, b2, eps, wd = (torch.tensor(float(x), dtype=torch.float32).double().item() for x in (lr, b1, b2, eps, wd))
    g = g * factor
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    theta = theta - lr * ((m / (1 - b1 ** t)) / (torch.sqrt(v / (1 - b2 ** t)) + eps) + wd * theta)
    return theta, m, v
