"""The 8-bit integer operators and the gated feed-forward block on real work:
what each computes in plain torch operations, the calls a program makes of the
library, and the bytes and operations that one pass cannot do without.

A row quantised to 8 bits here is whole numbers q from -127 to 127 with one
float32 scale s, the row's largest magnitude over 127: its values are q s.

Kinds of case:

* ``cast``   a matrix is quantised along its rows and read back in its type;
* ``mm``     C = A.B^T of two such matrices, a scale for each row of A (token)
  and of B (channel);
* ``ffn``    a served feed-forward layer in 8 bits: the tokens are quantised,
  the gated block multiplies them, its 16-bit result is quantised and the down
  projection multiplies that;
* ``gated``  the gated block in 16 bits, H = act(X.Wg^T) (X.Wu^T), as a server
  runs it;
* ``step``   the same block in training: forward, keeping G = X.Wg^T and
  U = X.Wu^T in 16 bits, and backward from dH to dG, dU, dX, dWg and dWu.

An operator's result in 16 bits is rounded once; what follows it in a case
takes it as rounded.
"""
import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # one token's activations before an 8-bit layer: latency alone
        dict(name="cast-token", kind="cast", R=1, C=8192, type="bf16", tight=False),
        # a long batch's activations
        dict(name="cast-batch", kind="cast", R=8192, C=8192, type="bf16", tight=False),
        # one token through a square projection
        dict(name="mm-token", kind="mm", M=1, N=8192, K=8192, out="bf16", tight=False),
        # the benchmark's ragged product, rows packed without padding
        dict(name="mm-ragged", kind="mm", M=1000, N=1500, K=777, out="f32", tight=True),
        # the benchmark's large compute-bound product
        dict(name="mm-8192", kind="mm", M=8192, N=8192, K=8192, out="bf16", tight=False),
        # one token through a whole layer: four launches that follow each other
        dict(name="ffn-token", kind="ffn", T=1, I=4096, O=8192, type="bf16", act="silu"),
        # a prompt through a whole layer
        dict(name="ffn-prompt", kind="ffn", T=2048, I=4096, O=8192, type="bf16", act="silu"),
        # one token in decoding, weights in 16 bits: they are all there is to read
        dict(name="gated-token", kind="gated", M=1, N=8192, K=8192, type="bf16", act="silu", tight=False),
        # sixteen sequences in decoding
        dict(name="gated-16", kind="gated", M=16, N=8192, K=4096, type="f16", act="gelu", tight=False),
        # a long prompt
        dict(name="gated-prompt", kind="gated", M=4096, N=8192, K=8192, type="bf16", act="silu", tight=False),
        # one training step on 4096 tokens
        dict(name="step-4096", kind="step", M=4096, N=8192, K=4096, type="bf16", act="silu", tight=False),
        # one on a ragged batch through a layer of odd width
        dict(name="step-ragged", kind="step", M=1000, N=1500, K=777, type="f16", act="gelu_tanh", tight=True),
    ]


ACTS = ["silu", "silu", "gelu", "gelu_tanh", "relu", "none"]


def _size(rng, lo, hi):
    """A size between lo and hi, even over its logarithm; about half are whole multiples of 64."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if n >= 128 and rng.random() < 0.5:
        n = n // 64 * 64
    return max(lo, min(hi, n))


def draw(rng):
    kind = rng.choice(["cast", "mm", "mm", "mm", "ffn", "gated", "gated", "gated", "step", "step"])
    tight = rng.random() < 0.3
    while True:
        if kind == "cast":
            c = dict(kind=kind, R=_size(rng, 1, 16384), C=_size(rng, 32, 16384),
                     type=rng.choice(["f32", "bf16", "f16"]), tight=tight)
            if c["R"] * c["C"] <= 1 << 26:
                return c
        elif kind == "mm":
            c = dict(kind=kind, M=_size(rng, 1, 8192), N=_size(rng, 64, 16384), K=_size(rng, 32, 16384),
                     out=rng.choice(["f32", "bf16", "f16"]), tight=tight)
            if c["M"] * c["N"] * c["K"] <= 1 << 38:
                return c
        elif kind == "ffn":
            c = dict(kind=kind, T=_size(rng, 1, 4096), I=_size(rng, 64, 8192), O=_size(rng, 64, 16384),
                     type=rng.choice(["bf16", "f16"]), act=rng.choice(ACTS))
            if c["T"] * c["I"] * c["O"] <= 1 << 36:
                return c
        else:
            lo = 1 if kind == "gated" else 64
            c = dict(kind=kind, M=_size(rng, lo, 8192), N=_size(rng, 64, 16384), K=_size(rng, 64, 8192),
                     type=rng.choice(["bf16", "f16"]), act=rng.choice(ACTS), tight=tight)
            if c["M"] * c["N"] * c["K"] <= 1 << (37 if kind == "gated" else 36):
                return c


def work(case):
    k = case["kind"]
    if k == "cast":
        R, C, e = case["R"], case["C"], SIZE[case["type"]]
        return {"bytes": 2 * (e + 1) * R * C + 8 * R, "flops": 0}
    if k == "mm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + 4 * (M + N) + SIZE[case["out"]] * M * N, "flops": 2 * M * N * K}
    if k == "ffn":
        T, I, O = case["T"], case["I"], case["O"]
        cast = 3 * T * (I + O) + 8 * T
        mm = T * I + 2 * O * I + 4 * (T + 2 * O) + 2 * T * O + T * O + I * O + 4 * (T + I) + 2 * T * I
        return {"bytes": cast + mm, "flops": 6 * T * I * O}
    M, N, K = case["M"], case["N"], case["K"]
    forward = 2 * (M * K + 2 * N * K + M * N)
    if k == "gated":
        return {"bytes": forward, "flops": 4 * M * N * K}
    # G and U are written and read again, dG and dU written and read by each of the two products
    back = 2 * (2 * M * N + 3 * M * N + 2 * M * N) + 2 * (2 * M * N + 2 * N * K + M * K) + 2 * (2 * M * N + M * K + 2 * N * K)
    return {"bytes": forward + back, "flops": 12 * M * N * K}


# ---- the plain form --------------------------------------------------------

def _quantise(x):
    """(whole numbers, scales) of a matrix along its rows.  The quotient is taken in 64 bits: in 32 one
    next to a half could fall on it."""
    x = x.float()
    s = torch.clamp(x.abs().amax(1) / 127.0, min=2.0 ** -126)
    return torch.round(x.double() / s.double()[:, None]).float(), s


def _act(name, x):
    if name == "none":
        return x
    if name == "relu":
        return torch.where(x < 0, 0.0, x)
    if name == "silu":
        return x / (1 + torch.exp(-x))
    if name == "gelu":
        return 0.5 * x * torch.erfc(-x * math.sqrt(0.5))
    return x / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))


def _slope(name, x):
    """The activation's derivative."""
    if name == "none":
        return torch.ones_like(x)
    if name == "relu":
        return (x > 0).to(x.dtype)
    if name == "silu":
        s = 1 / (1 + torch.exp(-x))
        return s * (1 + x * (1 - s))
    if name == "gelu":
        return 0.5 * torch.erfc(-x * math.sqrt(0.5)) + x * torch.exp(-0.5 * x * x) * math.sqrt(0.5 / math.pi)
    c = math.sqrt(2 / math.pi)
    s = 1 / (1 + torch.exp(-2 * c * (x + 0.044715 * x * x * x)))
    return s + 2 * x * s * (1 - s) * c * (1 + 3 * 0.044715 * x * x)


def _product(a, sa, b, sb):
    return (a.float() @ b.float().t()) * sa[:, None] * sb


def _plain(st):
    k = st["kind"]
    if k == "cast":
        q, s = _quantise(st["X"])
        return (q * s[:, None]).to(st["X"].dtype)
    if k == "mm":
        return _product(st["A"], st["SA"], st["B"], st["SB"]).to(st["Y"].dtype)
    if k == "ffn":
        t = st["X"].dtype
        q, s = _quantise(st["X"])
        h = (_act(st["act"], _product(q, s, st["G"], st["SG"])) * _product(q, s, st["U"], st["SU"])).to(t)
        q, s = _quantise(h)
        return {"h": h, "y": _product(q, s, st["D"], st["SD"]).to(t)}
    t, x, wg, wu = st["X"].dtype, st["X"].float(), st["WG"].float(), st["WU"].float()
    g, u = x @ wg.t(), x @ wu.t()
    h = (_act(st["act"], g) * u).to(t)
    if k == "gated":
        return h
    out = {"h": h, "g": g.to(t), "u": u.to(t)}
    g, u, dh = out["g"].float(), out["u"].float(), st["DH"].float()
    dg, du = dh * u * _slope(st["act"], g), dh * _act(st["act"], g)
    out.update(dg=dg.to(t), du=du.to(t))
    out.update(dx=(dg @ wg + du @ wu).to(t), dwg=(dg.t() @ x).to(t), dwu=(du.t() @ x).to(t))
    return out


# ---- inputs ----------------------------------------------------------------

def _padded(rows, cols, dtype, tight):
    """An empty matrix whose rows are packed, or begin on whole 16 bytes."""
    n = 16 // torch.empty((), dtype=dtype).element_size()
    ld = cols if tight else -(-cols // n) * n
    return torch.zeros((rows, ld), dtype=dtype, device=DEVICE)[:, :cols]


def _into(x, dtype, tight):
    y = _padded(x.shape[0], x.shape[1], dtype, tight)
    y.copy_(x)
    return y


def _activations(gen, rows, cols):
    """Normal values with a few outlying channels, and rows of zeros behind a batch's last token."""
    x = torch.randn((rows, cols), generator=gen, device=DEVICE)
    x *= torch.exp(0.5 * torch.randn((1, cols), generator=gen, device=DEVICE))
    x *= torch.where(torch.rand((1, cols), generator=gen, device=DEVICE) < 0.01, 20.0, 1.0)
    if rows >= 16:
        x[rows - rows // 16:] = 0
    return x


def _weights(gen, rows, cols):
    return 0.02 * torch.randn((rows, cols), generator=gen, device=DEVICE)


def _gradients(gen, rows, cols, dtype):
    """Small values whose size differs from token to token; scaled up where the type's range is short."""
    x = (1e-1 if dtype == torch.float16 else 1e-4) * torch.randn((rows, cols), generator=gen, device=DEVICE)
    return x * torch.exp(torch.randn((rows, 1), generator=gen, device=DEVICE))


def _int8(x, tight):
    q, s = _quantise(x)
    return _into(q, torch.int8, tight), s


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed) * 2654435761 % (1 << 62) + 29)
    st = dict(case)
    k = case["kind"]
    if k == "cast":
        R, C, t = case["R"], case["C"], TYPES[case["type"]]
        x = _weights(gen, R, C) if case["type"] == "f32" else _activations(gen, R, C)
        st["X"], st["Y"] = _into(x, t, case["tight"]), _padded(R, C, t, case["tight"])
        st["Q"] = _padded(R, C, torch.int8, case["tight"])
        st["S"] = torch.empty(R, device=DEVICE)
    elif k == "mm":
        M, N, K, tight = case["M"], case["N"], case["K"], case["tight"]
        st["A"], st["SA"] = _int8(_activations(gen, M, K), tight)
        st["B"], st["SB"] = _int8(_weights(gen, N, K), tight)
        st["Y"] = _padded(M, N, TYPES[case["out"]], tight)
    elif k == "ffn":
        T, I, O, t = case["T"], case["I"], case["O"], TYPES[case["type"]]
        st["X"] = _into(_activations(gen, T, I), t, False)
        st["G"], st["SG"] = _int8(_weights(gen, O, I), False)
        st["U"], st["SU"] = _int8(_weights(gen, O, I), False)
        st["D"], st["SD"] = _int8(_weights(gen, I, O), False)
        st["Q"], st["S"] = _padded(T, I, torch.int8, False), torch.empty(T, device=DEVICE)
        st["H"] = _padded(T, O, t, False)
        st["HQ"], st["HS"] = _padded(T, O, torch.int8, False), torch.empty(T, device=DEVICE)
        st["Y"] = _padded(T, I, t, False)
    else:
        M, N, K, t, tight = case["M"], case["N"], case["K"], TYPES[case["type"]], case["tight"]
        st["X"] = _into(_activations(gen, M, K), t, tight)
        st["WG"] = _into(_weights(gen, N, K), t, tight)
        st["WU"] = _into(_weights(gen, N, K), t, tight)
        st["H"] = _padded(M, N, t, tight)
        if k == "step":
            st["DH"] = _into(_gradients(gen, M, N, t), t, tight)
            for name, (r, c) in {"G": (M, N), "U": (M, N), "DG": (M, N), "DU": (M, N), "DX": (M, K),
                                 "DWG": (N, K), "DWU": (N, K)}.items():
                st[name] = _padded(r, c, t, tight)
    return st


# ---- the framework's calls -------------------------------------------------

def _named(b, name, x):
    return getattr(b, name + {torch.float32: "_f32", torch.bfloat16: "_bf16", torch.float16: "_f16"}[x.dtype])


def _cast(b, x, q, s):
    _named(b, "gemm_i8_quantize", x)(x.shape[0], x.shape[1], x, x.stride(0), q, q.stride(0), s)


def _mm(b, a, sa, w, sw, y):
    _named(b, "gemm_i8", y)(y.shape[0], y.shape[1], a.shape[1], a, a.stride(0), sa, w, w.stride(0), sw, y, y.stride(0))


def _calls(st):
    from register_lds_tiled_amd import binding as b
    k = st["kind"]
    if k == "cast":
        q, y = st["Q"], st["Y"]
        _cast(b, st["X"], q, st["S"])
        _named(b, "gemm_i8_dequantize", y)(y.shape[0], y.shape[1], q, q.stride(0), st["S"], y, y.stride(0))
        return y
    if k == "mm":
        _mm(b, st["A"], st["SA"], st["B"], st["SB"], st["Y"])
        return st["Y"]
    if k == "ffn":
        q, g, u, h = st["Q"], st["G"], st["U"], st["H"]
        _cast(b, st["X"], q, st["S"])
        _named(b, "gemm_i8_gated", h)(h.shape[0], h.shape[1], q.shape[1], q, q.stride(0), st["S"], g, g.stride(0), st["SG"],
                                      u, u.stride(0), st["SU"], h, h.stride(0), st["act"])
        _cast(b, h, st["HQ"], st["HS"])
        _mm(b, st["HQ"], st["HS"], st["D"], st["SD"], st["Y"])
        return {"h": h, "y": st["Y"]}
    x, wg, wu, h = st["X"], st["WG"], st["WU"], st["H"]
    M, N, K = st["M"], st["N"], st["K"]
    at = lambda *names: [v for n in names for v in (st[n], st[n].stride(0))]  # noqa: E731
    if k == "gated":
        _named(b, "gemm_gated", h)(M, N, K, *at("X", "WG", "WU"), None, 0, None, 0, *at("H"), st["act"])
        return h
    _named(b, "gemm_gated", h)(M, N, K, *at("X", "WG", "WU", "G", "U", "H"), st["act"])
    _named(b, "gemm_gated_backward", h)(M, N, K, *at("X", "WG", "WU", "G", "U", "DH", "DG", "DU", "DX", "DWG", "DWU"),
                                        st["act"])
    return {"h": h, "g": st["G"], "u": st["U"], "dg": st["DG"], "du": st["DU"], "dx": st["DX"],
            "dwg": st["DWG"], "dwu": st["DWU"]}


def run(state):
    return _calls(state) if own else _plain(state)


# ---- the definition in 64 bits ---------------------------------------------

def _cast64(x):
    """(whole numbers, scales) in 64 bits: the scale is a float32, and a value goes to the whole number
    whose distance is less than half, to the even one of two as near."""
    x = x.double()
    s = torch.maximum((x.abs().max(1).values / 127).float().double(), torch.tensor(2.0 ** -126, dtype=torch.float64, device=x.device))
    r = x / s[:, None]
    low = torch.floor(r)
    up = (r - low > 0.5) | ((r - low == 0.5) & (low % 2 == 1))
    return low + up, s


def _act64(name, x):
    """(activation, derivative), from sigmoid, tanh and the normal distribution's density and integral."""
    if name == "none":
        return x, torch.ones_like(x)
    if name == "relu":
        return x.clamp(min=0), torch.heaviside(x, torch.zeros((), dtype=x.dtype, device=x.device))
    if name == "silu":
        s = torch.sigmoid(x)
        return x * s, s + x * s * torch.sigmoid(-x)
    if name == "gelu":
        p = torch.special.ndtr(x)
        return x * p, p + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    y = math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
    t = torch.tanh(y)
    return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 0.134145 * x * x)


def exact(case, seed):
    st = prepare(case, seed)
    k = case["kind"]
    if k == "cast":
        q, s = _cast64(st["X"])
        return q * s[:, None]
    if k == "mm":
        return (st["A"].double() * st["SA"].double()[:, None]) @ (st["B"].double() * st["SB"].double()[:, None]).t()
    if k == "ffn":
        q, s = _cast64(st["X"])
        x = q * s[:, None]
        g = x @ (st["G"].double() * st["SG"].double()[:, None]).t()
        u = x @ (st["U"].double() * st["SU"].double()[:, None]).t()
        h = _act64(case["act"], g)[0] * u
        q, s = _cast64(h.to(st["X"].dtype))
        return {"h": h, "y": (q * s[:, None]) @ (st["D"].double() * st["SD"].double()[:, None]).t()}
    x, wg, wu = st["X"].double(), st["WG"].double(), st["WU"].double()
    g, u = x @ wg.t(), x @ wu.t()
    h = _act64(case["act"], g)[0] * u
    if k == "gated":
        return h
    a, d = _act64(case["act"], g.to(st["X"].dtype).double())
    dh = st["DH"].double()
    dg, du = dh * u.to(st["X"].dtype).double() * d, dh * a
    return {"h": h, "g": g, "u": u, "dg": dg, "du": du, "dx": dg @ wg + du @ wu, "dwg": dg.t() @ x, "dwu": du.t() @ x}
