"""The microscaled 4-bit operators on real work: what each computes in plain
torch operations, the calls a program makes of the library, and the bytes and
operations that one pass cannot do without.

MXFP4 here is: blocks of 32 consecutive values along a row share one scale
2^(s - 127), held as the byte s (255: the block is NaN), and each value is
four bits, sign, two exponent bits and one mantissa bit: 0, 0.5, 1, 1.5, 2, 3,
4, 6 and their negatives.  Two values to a byte, the even one in the low half;
a row of K values takes ceil(K / 2) bytes and ceil(K / 32) scales.

Kinds of case:

* ``cast``  a matrix is quantised (along its rows; where ``both``, along its
  columns too, into the transposed matrix that a backward pass multiplies
  with) and read back in its own type;
* ``mm``    C = A.B^T, both operands in MXFP4, as a layer multiplies once its
  activations are quantised;
* ``step``  a linear layer's training step: X, W and dY are quantised along
  both of their axes, and Y = X.W^T, dX = dY.W and dW = dY^T.X are multiplied;
* ``wo``    C = A.W^T with 16-bit activations and MXFP4 weights, as a server
  runs a model whose weights alone are quantised.
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
        # one token's activations before a quantised layer: latency alone
        dict(name="cast-token", kind="cast", R=1, C=8192, type="bf16", both=False, tight=False),
        # a training batch's activations, for the forward and the weight gradient
        dict(name="cast-activations", kind="cast", R=8192, C=8192, type="bf16", both=True, tight=False),
        # master weights kept in 32 bits, quantised after an optimiser step
        dict(name="cast-weights", kind="cast", R=16384, C=8192, type="f32", both=False, tight=False),
        # a ragged piece with rows of odd length, packed without padding
        dict(name="cast-ragged", kind="cast", R=1000, C=777, type="f16", both=True, tight=True),
        # one token through a square projection
        dict(name="mm-token", kind="mm", M=1, N=8192, K=8192, out="f32", tight=False),
        # the benchmark's ragged product
        dict(name="mm-ragged", kind="mm", M=1000, N=1500, K=777, out="f32", tight=True),
        # a prompt of 2048 tokens through a small projection
        dict(name="mm-2048", kind="mm", M=2048, N=2048, K=2048, out="bf16", tight=False),
        # the benchmark's large compute-bound product
        dict(name="mm-8192", kind="mm", M=8192, N=8192, K=8192, out="f32", tight=False),
        # one training step of a linear layer on 4096 tokens
        dict(name="step-4096", kind="step", T=4096, I=4096, O=8192),
        # one token in decoding: the weights are all there is to read
        dict(name="wo-token", kind="wo", M=1, N=8192, K=8192, type="bf16", tight=False),
        # sixteen sequences through an output layer as wide as a vocabulary
        dict(name="wo-16", kind="wo", M=16, N=65536, K=8192, type="f16", tight=False),
        # a long prompt with weights in four bits
        dict(name="wo-prompt", kind="wo", M=4096, N=8192, K=8192, type="bf16", tight=False),
    ]


def _size(rng, lo, hi):
    """A size between lo and hi, even over its logarithm; about half are whole multiples of 64."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if n >= 128 and rng.random() < 0.5:
        n = n // 64 * 64
    return max(lo, min(hi, n))


def draw(rng):
    kind = rng.choice(["cast", "cast", "mm", "mm", "mm", "step", "wo", "wo", "wo"])
    tight = rng.random() < 0.3
    while True:
        if kind == "cast":
            c = dict(kind=kind, R=_size(rng, 1, 16384), C=_size(rng, 32, 16384),
                     type=rng.choice(["f32", "bf16", "f16"]), both=rng.random() < 0.5, tight=tight)
            if c["R"] * c["C"] <= (1 << 27 if not c["both"] else 1 << 26):
                return c
        elif kind == "mm":
            c = dict(kind=kind, M=_size(rng, 1, 8192), N=_size(rng, 64, 16384), K=_size(rng, 32, 16384),
                     out=rng.choice(["f32", "bf16"]), tight=tight)
            if c["M"] * c["N"] * c["K"] <= 1 << 37:
                return c
        elif kind == "step":
            c = dict(kind=kind, T=_size(rng, 64, 8192), I=_size(rng, 64, 8192), O=_size(rng, 64, 8192))
            if c["T"] * c["I"] * c["O"] <= 1 << 37:
                return c
        else:
            c = dict(kind=kind, M=_size(rng, 1, 4096), N=_size(rng, 64, 65536), K=_size(rng, 32, 8192),
                     type=rng.choice(["bf16", "f16"]), tight=tight)
            if c["M"] * c["N"] * c["K"] <= 1 << 38 and c["N"] * c["K"] <= 1 << 29:
                return c


def _packed(rows, k):
    """Bytes of an MXFP4 matrix: its values and its scales."""
    return rows * (-(-k // 2) + -(-k // 32))


def work(case):
    k = case["kind"]
    if k == "cast":
        R, C, e = case["R"], case["C"], SIZE[case["type"]]
        n = e * R * C + 2 * _packed(R, C) + e * R * C      # quantised, and read back
        if case["both"]:
            n += 2 * _packed(C, R) + e * R * C
        return {"bytes": n, "flops": 0}
    if k == "step":
        T, I, O = case["T"], case["I"], case["O"]
        cast = sum(2 * r * c + _packed(r, c) + _packed(c, r) for r, c in ((T, I), (O, I), (T, O)))
        mm = (_packed(T, I) + _packed(O, I) + 2 * T * O + _packed(T, O) + _packed(I, O) + 2 * T * I
              + _packed(O, T) + _packed(I, T) + 4 * O * I)
        return {"bytes": cast + mm, "flops": 6 * T * I * O}
    M, N, K = case["M"], case["N"], case["K"]
    if k == "mm":
        return {"bytes": _packed(M, K) + _packed(N, K) + SIZE[case["out"]] * M * N, "flops": 2 * M * N * K}
    return {"bytes": 2 * M * K + _packed(N, K) + 4 * M * N, "flops": 2 * M * N * K}


# ---- the plain form --------------------------------------------------------

def _blocks(x):
    """x (rows x K, float32) as rows x blocks x 32, zeros behind the last value."""
    rows, k = x.shape
    nb = -(-k // 32)
    if nb * 32 != k:
        x = torch.nn.functional.pad(x, (0, nb * 32 - k))
    return x.reshape(rows, nb, 32)


def _scaled(x, n):
    """x 2^n, n whole numbers of at most 252 either way, in two steps by powers of two made from their bits
    (a library's power is an ulp off here and there, which would tip ties)."""
    h = torch.div(n, 2, rounding_mode="floor")
    return x * ((h + 127) << 23).view(torch.float32) * ((n - h + 127) << 23).view(torch.float32)


def _quantise(x):
    """(codes, scales) of a matrix along its rows: codes rows x K, one to a byte, scales rows x blocks.

    The scale's exponent is the largest magnitude's, less 2 (that of the format's largest value); a value
    is rounded to the nearest, ties to the even code, and past the largest to the largest."""
    rows, k = x.shape
    b = _blocks(x.float().contiguous())
    top = b.abs().amax(-1)
    e = torch.frexp(top).exponent - 3
    s = torch.where(top > 0, e, -127).clamp(min=-127).int()
    a = _scaled(b, -s[..., None]).abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp(max=6.0)
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code + (torch.signbit(b).to(torch.uint8) << 3)
    bad = ~torch.isfinite(top)
    scale = torch.where(bad, 255, s + 127).to(torch.uint8)
    return code.reshape(rows, -1)[:, :k], scale


def _pack(code, ld):
    """Codes two to a byte, the even one low, rows ld bytes apart."""
    rows, k = code.shape
    if k % 2:
        code = torch.nn.functional.pad(code, (0, 1))
    q = torch.zeros((rows, ld), dtype=torch.uint8, device=code.device)
    q[:, :code.shape[1] // 2] = code[:, 0::2] | (code[:, 1::2] << 4)
    return q


def _values(code, scale):
    """The float32 values of codes (rows x K) with their scales (rows x blocks)."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=code.device)
    table = torch.cat([table, -table])
    k = code.shape[1]
    f = torch.where(scale == 255, torch.full((), float("nan"), device=scale.device),
                    _scaled(torch.ones((), device=scale.device), scale.int() - 127))
    return table[code.int()] * f.repeat_interleave(32, 1)[:, :k]


def _unpack(q, k):
    """The codes, one to a byte, of k values a row."""
    return torch.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1)[:, :k]


def _plain(st):
    k = st["kind"]
    if k == "cast":
        x = st["X"]
        out = {"rows": _values(*_quantise(x)).to(x.dtype)}
        if st["both"]:
            out["cols"] = _values(*_quantise(x.t())).to(x.dtype)
        return out
    if k == "mm":
        a = _values(_unpack(st["A"], st["K"]), st["SA"])
        b = _values(_unpack(st["B"], st["K"]), st["SB"])
        return (a @ b.t()).to(st["Y"].dtype)
    if k == "wo":
        w = _values(_unpack(st["B"], st["K"]), st["SB"])
        return st["A"].float() @ w.t()
    x, w, g = st["X"], st["W"], st["G"]
    y = _values(*_quantise(x)) @ _values(*_quantise(w)).t()
    dx = _values(*_quantise(g)) @ _values(*_quantise(w.t())).t()
    dw = _values(*_quantise(g.t())) @ _values(*_quantise(x.t())).t()
    return {"y": y.to(torch.bfloat16), "dx": dx.to(torch.bfloat16), "dw": dw}


# ---- inputs ----------------------------------------------------------------

def _activations(gen, rows, cols, dtype):
    """Normal values with a few outlying channels, and rows of zeros behind a batch's last token."""
    x = torch.randn((rows, cols), generator=gen, device=DEVICE)
    x *= torch.exp(0.5 * torch.randn((1, cols), generator=gen, device=DEVICE))
    x *= torch.where(torch.rand((1, cols), generator=gen, device=DEVICE) < 0.01, 20.0, 1.0)
    if rows >= 16:
        x[rows - rows // 16:] = 0
    return x.to(dtype)


def _weights(gen, rows, cols, dtype):
    return (0.02 * torch.randn((rows, cols), generator=gen, device=DEVICE)).to(dtype)


def _gradients(gen, rows, cols, dtype):
    """Small values whose size differs from token to token."""
    x = 1e-4 * torch.randn((rows, cols), generator=gen, device=DEVICE)
    return (x * torch.exp(torch.randn((rows, 1), generator=gen, device=DEVICE))).to(dtype)


def _ld(k, tight):
    """Bytes from row to row: what k values take, or that in whole 16 bytes."""
    n = max(1, -(-k // 2))
    return n if tight else -(-n // 16) * 16


def _room(rows, k, tight=False):
    """An MXFP4 matrix's buffers, as a program holds them before they are filled."""
    return (torch.empty((rows, _ld(k, tight)), dtype=torch.uint8, device=DEVICE),
            torch.empty((rows, -(-k // 32)), dtype=torch.uint8, device=DEVICE))


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)
    st = dict(case)
    k = case["kind"]
    if k == "cast":
        R, C, t = case["R"], case["C"], TYPES[case["type"]]
        st["X"] = _weights(gen, R, C, t) if case["type"] == "f32" else _activations(gen, R, C, t)
        st["Q"], st["S"] = _room(R, C, case["tight"])
        st["Y"] = torch.empty((R, C), dtype=t, device=DEVICE)
        if case["both"]:
            st["QT"], st["ST"] = _room(C, R, case["tight"])
            st["YT"] = torch.empty((C, R), dtype=t, device=DEVICE)
    elif k == "step":
        T, I, O = case["T"], case["I"], case["O"]
        st["X"] = _activations(gen, T, I, torch.bfloat16)
        st["W"] = _weights(gen, O, I, torch.bfloat16)
        st["G"] = _gradients(gen, T, O, torch.bfloat16)
        for name, (r, c) in {"X": (T, I), "W": (O, I), "G": (T, O)}.items():
            st[name + "q"], st[name + "s"] = _room(r, c)
            st[name + "qt"], st[name + "st"] = _room(c, r)
        st["y"] = torch.empty((T, O), dtype=torch.bfloat16, device=DEVICE)
        st["dx"] = torch.empty((T, I), dtype=torch.bfloat16, device=DEVICE)
        st["dw"] = torch.empty((O, I), dtype=torch.float32, device=DEVICE)
    else:
        M, N, K = case["M"], case["N"], case["K"]
        code, st["SB"] = _quantise(_weights(gen, N, K, torch.float32))
        st["B"] = _pack(code, _ld(K, case["tight"]))
        if k == "mm":
            code, st["SA"] = _quantise(_activations(gen, M, K, torch.bfloat16))
            st["A"] = _pack(code, _ld(K, case["tight"]))
            st["Y"] = torch.empty((M, N), dtype=TYPES[case["out"]], device=DEVICE)
        else:
            st["A"] = _activations(gen, M, K, TYPES[case["type"]])
            st["Y"] = torch.empty((M, N), dtype=torch.float32, device=DEVICE)
    return st


# ---- the framework's calls -------------------------------------------------

def _cast(b, x, q, s, qt=None, st=None):
    f = {torch.float32: b.gemm_mxfp4_quantize_f32, torch.bfloat16: b.gemm_mxfp4_quantize_bf16,
         torch.float16: b.gemm_mxfp4_quantize_f16}[x.dtype]
    f(x.shape[0], x.shape[1], x, x.stride(0), q, 0 if q is None else q.stride(0), s, 0 if s is None else s.stride(0),
      qt, 0 if qt is None else qt.stride(0), st, 0 if st is None else st.stride(0))


def _back(b, q, s, y):
    f = {torch.float32: b.gemm_mxfp4_dequantize_f32, torch.bfloat16: b.gemm_mxfp4_dequantize_bf16,
         torch.float16: b.gemm_mxfp4_dequantize_f16}[y.dtype]
    f(y.shape[0], y.shape[1], q, q.stride(0), s, s.stride(0), y, y.stride(0))


def _mm(b, k, a, sa, w, sw, c):
    f = {torch.float32: b.gemm_mxfp4_f32, torch.bfloat16: b.gemm_mxfp4_bf16}[c.dtype]
    f(c.shape[0], c.shape[1], k, a, a.stride(0), sa, sa.stride(0), w, w.stride(0), sw, sw.stride(0), c, c.stride(0))


def _calls(st):
    from register_lds_tiled_amd import binding as b
    k = st["kind"]
    if k == "cast":
        _cast(b, st["X"], st["Q"], st["S"], st.get("QT"), st.get("ST"))
        _back(b, st["Q"], st["S"], st["Y"])
        out = {"rows": st["Y"]}
        if st["both"]:
            _back(b, st["QT"], st["ST"], st["YT"])
            out["cols"] = st["YT"]
        return out
    if k == "mm":
        _mm(b, st["K"], st["A"], st["SA"], st["B"], st["SB"], st["Y"])
        return st["Y"]
    if k == "wo":
        a, w, s, y = st["A"], st["B"], st["SB"], st["Y"]
        f = b.gemm_bf16_mxfp4_f32 if a.dtype == torch.bfloat16 else b.gemm_f16_mxfp4_f32
        f(st["M"], st["N"], st["K"], a, a.stride(0), w, w.stride(0), s, s.stride(0), y, y.stride(0))
        return y
    for n in ("X", "W", "G"):
        _cast(b, st[n], st[n + "q"], st[n + "s"], st[n + "qt"], st[n + "st"])
    _mm(b, st["I"], st["Xq"], st["Xs"], st["Wq"], st["Ws"], st["y"])
    _mm(b, st["O"], st["Gq"], st["Gs"], st["Wqt"], st["Wst"], st["dx"])
    _mm(b, st["T"], st["Gqt"], st["Gst"], st["Xqt"], st["Xst"], st["dw"])
    return {"y": st["y"], "dx": st["dx"], "dw": st["dw"]}


def run(state):
    return _calls(state) if own else _plain(state)


# ---- the definition in 64 bits ---------------------------------------------

def _two_to(n):
    """2^n in 64 bits, from its bits."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _cast64(x):
    """The values a matrix has once quantised along its rows, by counting the borders each magnitude passes."""
    rows, k = x.shape
    nb = -(-k // 32)
    b = torch.zeros((rows, nb * 32), dtype=torch.float64, device=x.device)
    b[:, :k] = x.double()
    b = b.view(rows, nb, 32)
    top = b.abs().max(-1, keepdim=True).values
    scale = _two_to(torch.clamp(torch.floor(torch.log2(top)) - 2, min=-127.0))
    m = b.abs() / scale
    # a value is the sum of the steps whose border it has passed; a border itself goes to the even code
    v = 0.5 * (m > 0.25) + 0.5 * (m >= 0.75) + 0.5 * (m > 1.25) + 0.5 * (m >= 1.75)
    v = v + (m > 2.5) + (m >= 3.5) + 2.0 * (m > 5.0)
    return (v * torch.sign(b) * scale).view(rows, nb * 32)[:, :k]


def _decode64(q, s, k):
    """The values of a packed matrix from the bits: (-1)^sign 2^(e - 1) (1 + m / 2), and m / 2 where e is 0."""
    n = torch.arange(k, device=q.device)
    c = (q.long()[:, n // 2] >> (4 * (n % 2))) & 15
    e, m = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e == 0, m / 2, (1 + m / 2) * _two_to(e - 1))
    v = torch.where(c >= 8, -v, v)
    return v * _two_to(s.long() - 127)[:, n // 32]


def exact(case, seed):
    st = prepare(case, seed)
    k = case["kind"]
    if k == "cast":
        out = {"rows": _cast64(st["X"])}
        if case["both"]:
            out["cols"] = _cast64(st["X"].t())
        return out
    if k == "mm":
        return _decode64(st["A"], st["SA"], case["K"]) @ _decode64(st["B"], st["SB"], case["K"]).t()
    if k == "wo":
        return st["A"].double() @ _decode64(st["B"], st["SB"], case["K"]).t()
    x, w, g = st["X"], st["W"], st["G"]
    return {"y": _cast64(x) @ _cast64(w).t(), "dx": _cast64(g) @ _cast64(w.t()).t(),
            "dw": _cast64(g.t()) @ _cast64(x.t()).t()}
