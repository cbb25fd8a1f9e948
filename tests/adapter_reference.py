"""Plain fp64 restatement of the adapter operators, and fp32 / fp64 ones of the AdamW step,
written from the formulas for the tests (no code shared with the library)."""
import math

import numpy as np
import torch

U16 = 2.0 ** -11  # half a step of fp16, relative
U32 = 2.0 ** -24


class Pool:
    """Adapters of one projection shape as the test sees them: fp16 weights, ranks, scales."""

    def __init__(self, d_in, d_out, max_rank, ranks, seed=0, scale=None):
        g = torch.Generator().manual_seed(seed)
        self.d_in, self.d_out, self.max_rank, self.ranks = d_in, d_out, max_rank, list(ranks)
        self.A = [(torch.randn(r, d_in, generator=g) * d_in ** -0.5).half().cuda() for r in self.ranks]
        self.B = [(torch.randn(r, d_out, generator=g) * 0.1).half().cuda() for r in self.ranks]
        self.scale = [float(np.float32(1.0 + 0.37 * (i % 5))) if scale is None else scale for i in range(len(self.ranks))]

    def upload(self, dp, max_tokens, stream=0):
        h = dp.dictproj_adapters_create(self.d_in, self.d_out, self.max_rank, len(self.ranks), max_tokens)
        for s, r in enumerate(self.ranks):
            dp.dictproj_adapters_set(h, s, r, self.scale[s], self.A[s].data_ptr() if r else 0,
                                     self.B[s].data_ptr() if r else 0, stream)
        return h


def rows_of(ids, slot):
    return torch.nonzero(ids == slot).flatten()


def forward(pool, ids, X, base=None):
    """(Y, W) in fp64: the result and the sum of the absolute values of its adapter terms."""
    Y = torch.zeros(X.shape[0], pool.d_out, dtype=torch.float64, device="cuda") if base is None else base.double()
    W = torch.zeros_like(Y)
    for s, r in enumerate(pool.ranks):
        at = rows_of(ids, s)
        if r == 0 or at.numel() == 0:
            continue
        x, a, b, w = X[at].double(), pool.A[s].double(), pool.B[s].double(), pool.scale[s]
        Y[at] += w * ((x @ a.T) @ b)
        W[at] += abs(w) * ((x.abs() @ a.abs().T) @ b.abs())
    return Y, W


def backward(pool, ids, X, dY, base=None):
    """fp64 {'dX', 'dA', 'dB'} and the sums of absolute values {'WX', 'WA', 'WB'}."""
    n, R = len(pool.ranks), pool.max_rank
    z = lambda *s: torch.zeros(*s, dtype=torch.float64, device="cuda")  # noqa: E731
    o = {"dX": z(X.shape[0], pool.d_in) if base is None else base.double(), "dA": z(n, R, pool.d_in),
         "dB": z(n, R, pool.d_out), "WX": z(X.shape[0], pool.d_in), "WA": z(n, R, pool.d_in), "WB": z(n, R, pool.d_out)}
    for s, r in enumerate(pool.ranks):
        at = rows_of(ids, s)
        if r == 0 or at.numel() == 0:
            continue
        x, y, a, b, w = X[at].double(), dY[at].double(), pool.A[s].double(), pool.B[s].double(), pool.scale[s]
        u, t = w * (y @ b.T), w * (x @ a.T)
        ua, ta = abs(w) * (y.abs() @ b.abs().T), abs(w) * (x.abs() @ a.abs().T)
        o["dX"][at] += u @ a
        o["WX"][at] += ua @ a.abs()
        o["dA"][s, :r], o["WA"][s, :r] = u.T @ x, ua.T @ x.abs()
        o["dB"][s, :r], o["WB"][s, :r] = t.T @ y, ta.T @ y.abs()
    return o


def assert_half(got, want, absolute, terms, what=""):
    """An fp16 result rounded once from fp32 sums of `terms` terms whose absolute values add up to
    `absolute`. Element by element: half a step of the result (2^-11, or 2^-25 among the subnormals),
    plus the worst case of the sums, one rounding of at most 2^-23 of the running sum per term. Over
    all elements: a rounding's mean square is at most a third of its bound's square, the sums' errors
    are a random walk (terms^1/2 roundings, a factor 4 of room)."""
    got, err = got.double(), (got.double() - want).abs()
    bound = U16 * want.abs() + 2.0 ** -25 + 2 * U32 * terms * absolute
    worst = (err / bound).max().item()
    assert worst <= 1.0, f"{what}: element error {worst:.3f} of its bound"
    if want.numel() >= 1024:
        norm = want.norm().item()
        limit = U16 / math.sqrt(3) * 1.05 * norm + 4 * 2 * U32 * math.sqrt(terms) * want.norm().item() + 2.0 ** -25 * math.sqrt(want.numel())
        assert err.norm().item() <= limit, f"{what}: error norm {err.norm().item():.3e} over {limit:.3e}"


def assert_float(got, want, absolute, terms, what=""):
    """An fp32 sum of `terms` terms: the same bounds with fp32's half step."""
    assert got.dtype == torch.float32
    err = (got.double() - want).abs()
    bound = 2 * U32 * (terms + 4) * absolute
    assert (err <= bound).all(), f"{what}: element error {(err / bound.clamp_min(1e-300)).max().item():.3f} of its bound"
    if want.numel() >= 1024 and want.norm() > 0:
        limit = 4 * 2 * U32 * math.sqrt(terms) * want.norm().item()
        assert err.norm().item() <= limit, f"{what}: error norm {err.norm().item():.3e} over {limit:.3e}"


# ---------------------------------------------------------------------------- AdamW
def e4m3_value(codes):
    return torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn).float().numpy()


def e4m3_nearest(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def dither(n, step):
    m = np.uint64(0xFFFFFFFF)
    h = (np.arange(n, dtype=np.uint64) * np.uint64(0x9E3779B9) + np.uint64(step * 0x6A09E667 & 0xFFFFFFFF)) & m
    h = ((h ^ (h >> np.uint64(16))) * np.uint64(0xBB67AE85)) & m
    h = ((h ^ (h >> np.uint64(15))) * np.uint64(0x6A09E667)) & m
    return (h >> np.uint64(12)).astype(np.uint32)


def _blocks(x):
    n = x.size
    return np.pad(x, (0, -n % 128)).reshape(-1, 128)


def _scale(x):
    return np.maximum(np.abs(_blocks(x)).max(axis=1) * (np.float32(1) / np.float32(448)), np.float32(2.0 ** -126)).astype(np.float32)


def each(scale, n):
    return np.repeat(scale, 128)[:n]


def adamw(t, step, lr, beta1, beta2, eps, weight_decay, grad_scale, bits):
    """One step of {'p','g','m','v'[,'m_scale','v_scale']} (numpy) in the stated fp32 order; a new dict."""
    f = np.float32
    p, n = t["p"], t["p"].size
    if bits == 8:
        m = e4m3_value(t["m"]) * each(t["m_scale"], n)
        r = e4m3_value(t["v"]) * each(t["v_scale"], n)
        v = r * r
    else:
        m, v = t["m"], t["v"]
    g = t["g"] * f(grad_scale)
    m = m * f(beta1) + g * f(1.0 - beta1)
    v = v * f(beta2) + (g * f(1.0 - beta2)) * g
    r = np.sqrt(v)
    d = r * f(1.0 / math.sqrt(1.0 - beta2 ** step)) + f(eps)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        p = p * f(1.0 - lr * weight_decay) - (m / d) * f(lr / (1.0 - beta1 ** step))
        out = {"p": p, "g": t["g"], "copy": p.astype(np.float16)}
    if bits == 32:
        return {**out, "m": m, "v": v}
    out["m_scale"], out["v_scale"] = _scale(m), _scale(r)
    out["m"] = e4m3_nearest(m / each(out["m_scale"], n))
    x = ((r / each(out["v_scale"], n)) * f(2.0 ** -120)).astype(np.float32)
    code = np.minimum((x.view(np.uint32) + dither(n, step)) >> np.uint32(20), np.uint32(0x7E))
    out["v"] = np.where(r > 0, np.maximum(code, 1), code).astype(np.uint8)
    return out
