"""What is measured of a gated feed-forward block: its norm, its products and their gradients in
FP32, and the block in 8 bits.

Every case names an operator (``op``) and its sizes:

* ``norm``     -- root-mean-square norm with the residual's addition, to 8 bits with a scale per
                  row (``quant``) or to FP32; ``train`` adds the gradients of the rows and the
                  weight;
* ``quantize`` -- rows to 8 bits with a scale each, the activation's product first where there
                  is a gate;
* ``i8``       -- the product of 8-bit rows with 8-bit channels, scaled by row and channel;
* ``gated``    -- both projections, the activation and the product; ``train`` adds the gradients
                  of the rows and of both projections;
* ``block``    -- norm, product, activation, product and the residual's addition, in 8 bits.

``run`` computes the plain form (elementary torch operations; 64 bits where a value goes to the
nearest whole number, else 32) or, where ``own`` is true, calls the library.  8-bit outputs are
returned as the whole numbers they hold, their scales beside them.
"""
import math

import torch

own = False

F32, F64, I8 = torch.float32, torch.float64, torch.int8
EPS = 2.0 ** -17  # of the norm: the same in 32 and 64 bits
ACTIVATIONS = ("silu", "gelu", "gelu_tanh")


def listed():
    return [
        # one sequence being decoded: latency is all there is
        {"name": "norm one token", "op": "norm", "T": 1, "N": 4096, "residual": True, "quant": True, "pad": 0,
         "train": False},
        # a long prompt on its way to a product in 8 bits, the last rows padding
        {"name": "norm prompt", "op": "norm", "T": 4095, "N": 4096, "residual": True, "quant": True, "pad": 95,
         "train": False},
        # a training step of odd length: the residual stream, the normalised rows, and back
        {"name": "norm train", "op": "norm", "T": 2011, "N": 2048, "residual": True, "quant": False, "pad": 0,
         "train": True},
        # one token's activations between two products in 8 bits
        {"name": "quantize one token", "op": "quantize", "T": 1, "N": 4095, "act": "silu"},
        # a prompt's activations between two products in 8 bits
        {"name": "quantize prompt", "op": "quantize", "T": 2047, "N": 4096, "act": "silu"},
        # one sequence being decoded: the weights are read once
        {"name": "i8 one token", "op": "i8", "M": 1, "N": 4096, "K": 4096},
        # a batch of sequences being decoded, an odd number of channels
        {"name": "i8 decode batch", "op": "i8", "M": 37, "N": 4095, "K": 2048},
        # a long prompt: matrix-product bound
        {"name": "i8 prompt", "op": "i8", "M": 4096, "N": 4096, "K": 4096},
        # a batch of sequences being decoded in FP32
        {"name": "gated decode batch", "op": "gated", "T": 29, "N": 4096, "K": 2048, "act": "silu", "train": False},
        # a long prompt in FP32
        {"name": "gated prompt", "op": "gated", "T": 4096, "N": 4096, "K": 2048, "act": "silu", "train": False},
        # a training step
        {"name": "gated train", "op": "gated", "T": 2000, "N": 2048, "K": 1024, "act": "gelu_tanh", "train": True},
        # the whole block in 8 bits, as a model's layer runs it
        {"name": "block in 8 bits", "op": "block", "T": 515, "N": 2816, "K": 1024, "act": "silu"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the ranges above: row counts and widths spread over their logarithm and
    mostly odd, every option drawn, work below the largest listed case's."""
    op = rng.choice(["norm", "quantize", "i8", "gated", "block"])
    act = rng.choice(ACTIVATIONS)
    if op in ("norm", "quantize"):
        n = _log(rng, 64, 8192)
        t = _log(rng, 1, min(16384, (1 << 24) // n))
        if op == "quantize":
            return {"op": op, "T": t, "N": n, "act": rng.choice(["", act])}
        train = rng.random() < 0.4
        return {"op": op, "T": t, "N": n, "residual": rng.random() < 0.7, "quant": not train and rng.random() < 0.7,
                "pad": rng.choice([0, t // 9]), "train": train}
    if op == "i8":
        m, n, k = _log(rng, 1, 4096), _log(rng, 64, 8192), _log(rng, 64, 8192)
        while m * n * k > 1 << 35 or n * k > 1 << 25:
            n, k = (n * 3 // 4, k) if n > k else (n, k * 3 // 4)
        return {"op": op, "M": m, "N": n, "K": k}
    train = op == "gated" and rng.random() < 0.5
    t = _log(rng, 1, 2048 if train or op == "block" else 4096)
    n, k = _log(rng, 128, 4096), _log(rng, 128, 4096)
    while n * k > 1 << 23 or t * n * k > 1 << (32 if train else 34):
        n, k = (n * 3 // 4, k) if n > k else (n, k * 3 // 4)
    case = {"op": op, "T": t, "N": n, "K": k, "act": act}
    return case if op == "block" else {**case, "train": train}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _ld(n):
    """8-bit rows begin 16 bytes apart."""
    return -(-n // 16) * 16


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(1000003 * int(seed) + 29)
    rnd = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    empty = lambda *s: torch.empty(*s, dtype=F32, device=dev)  # noqa: E731
    bytes8 = lambda r, n: torch.zeros(r, _ld(n), dtype=I8, device=dev)  # noqa: E731
    rows8 = lambda r, n: torch.randint(-127, 128, (r, _ld(n)), generator=gen, device=dev, dtype=I8)  # noqa: E731
    # a residual stream: a few of its columns are much larger than the others
    stream = lambda t, n: rnd(t, n) * torch.exp(0.5 * rnd(n))  # noqa: E731
    st = {"case": case}
    op = case["op"]
    if op == "norm":
        T, N = case["T"], case["N"]
        st["x"] = stream(T, N)
        st["residual"] = stream(T, N) if case["residual"] else None
        st["weight"] = 1.0 + 0.2 * rnd(N)
        if case["pad"]:
            st["x"][T - case["pad"]:] = 0.0
            if case["residual"]:
                st["residual"][T - case["pad"]:] = 0.0
        st["sum"] = empty(T, N) if case["residual"] else None
        if case["quant"]:
            st["q"], st["scales"] = bytes8(T, N), empty(T)
        else:
            st["y"] = empty(T, N)
        if case["train"]:
            st["dy"], st["dsum"] = rnd(T, N), rnd(T, N) if case["residual"] else None
            st["dh"], st["dweight"] = empty(T, N), empty(N)
        return st
    if op == "quantize":
        T, N = case["T"], case["N"]
        st["x"] = stream(T, N)
        st["gate"] = 2.0 * rnd(T, N) if case["act"] else None
        st["q"], st["scales"] = bytes8(T, N), empty(T)
        return st
    if op == "i8":
        M, N, K = case["M"], case["N"], case["K"]
        st["A"], st["B"] = rows8(M, K), rows8(N, K)
        st["a_scales"] = torch.exp(0.3 * rnd(M)) / 127.0
        st["b_scales"] = torch.exp(0.2 * rnd(N)) / (127.0 * math.sqrt(K))
        st["C"] = empty(M, N)
        return st
    T, N, K = case["T"], case["N"], case["K"]
    if op == "gated":
        st["x"], st["G"], st["U"] = rnd(T, K), rnd(K, N) / math.sqrt(K), rnd(K, N) / math.sqrt(K)
        st["y"] = empty(T, N)
        if case["train"]:
            st["dy"], st["gate"], st["up"] = rnd(T, N), empty(T, N), empty(T, N)
            st["dx"], st["dG"], st["dU"] = empty(T, K), empty(K, N), empty(K, N)
        return st
    st["x"], st["residual"], st["weight"] = stream(T, K), stream(T, K), 1.0 + 0.2 * rnd(K)
    st["sum"] = empty(T, K)
    # gate's channels, then up's; the way back down
    st["B"], st["B2"] = rows8(2 * N, K), rows8(K, N)
    st["b_scales"] = torch.exp(0.2 * rnd(2 * N)) / (73.0 * math.sqrt(K))
    st["b2_scales"] = torch.exp(0.2 * rnd(K)) / (73.0 * math.sqrt(N))
    st["q"], st["scales"] = bytes8(T, K), empty(T)
    st["H"], st["q2"], st["scales2"] = empty(T, 2 * N), bytes8(T, N), empty(T)
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _plain_act(g, act):
    """act(g), in g's type."""
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    if act == "gelu":
        return g * 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
    return g / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _plain_act_slope(g, act):
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return s * (1.0 + g * (1.0 - s))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    c = 2.0 * math.sqrt(2.0 / math.pi)
    s = 1.0 / (1.0 + torch.exp(-c * (g + 0.044715 * g * g * g)))
    return s + g * s * (1.0 - s) * c * (1.0 + 0.134145 * g * g)


def _plain_quantize(v):
    """Whole numbers and scales of rows in 32 bits: which of two neighbours a value goes to is
    decided in 64."""
    most = v.abs().max(1).values.double()
    per = torch.where(most > 0, 127.0 / most, torch.zeros_like(most))
    return torch.round(v.double() * per.unsqueeze(1)).to(I8), (most / 127.0).to(F32)


def _plain_norm(x, residual, weight):
    h = x if residual is None else x + residual
    h64 = h.double()
    r = 1.0 / torch.sqrt((h64 * h64).mean(1, keepdim=True) + EPS)
    return h, (h64 * r * weight.double()).to(F32)


def _plain_norm_case(st, c):
    h, y = _plain_norm(st["x"], st["residual"], st["weight"])
    head = () if st["residual"] is None else (h,)
    if c["quant"]:
        return head + _plain_quantize(y)
    if not c["train"]:
        return head + (y,)
    r = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
    g = st["dy"] * st["weight"]
    dh = r * (g - h * (r * r * (g * h).mean(1, keepdim=True)))
    if st["dsum"] is not None:
        dh = dh + st["dsum"]
    return head + (y, dh, (st["dy"] * h * r).sum(0))


def _plain_gated_case(st, c):
    gate, up = st["x"] @ st["G"], st["x"] @ st["U"]
    a = _plain_act(gate, c["act"])
    if not c["train"]:
        return a * up
    dgate, dup = st["dy"] * up * _plain_act_slope(gate, c["act"]), st["dy"] * a
    dx = dgate @ st["G"].t() + dup @ st["U"].t()
    xt = st["x"].t()
    return a * up, dx, xt @ dgate, xt @ dup


def _plain_block(st, c):
    """The products in 64 bits: their results go to the nearest whole number next."""
    N, K = c["N"], c["K"]
    h, y = _plain_norm(st["x"], st["residual"], st["weight"])
    q, s = _plain_quantize(y)
    H = q.double() @ st["B"][:, :K].double().t() * s.double().unsqueeze(1) * st["b_scales"].double()
    H = H.to(F32)
    v = (_plain_act(H[:, :N].double(), c["act"]) * H[:, N:].double()).to(F32)
    q2, s2 = _plain_quantize(v)
    out = q2.float() @ st["B2"][:, :N].float().t() * s2.unsqueeze(1) * st["b2_scales"] + h
    return q, s, q2, s2, out


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own_act(g, act):
    return {"silu": g.SGEMM_ACT_SILU, "gelu": g.SGEMM_ACT_GELU, "gelu_tanh": g.SGEMM_ACT_GELU_TANH}[act]


def _own_space(st, size, *args):
    if "space" not in st:  # a program keeps its workspace
        st["space"] = torch.empty(max(256, size(*args)), dtype=torch.uint8, device="cuda")
    return st["space"]


def _own_norm_case(st, c):
    import fp32_gemm_03_amd as g
    T, N = c["T"], c["N"]
    head = () if st["residual"] is None else (st["sum"],)
    if c["quant"]:
        g.sgemm_norm(T, N, st["x"], N, st["residual"], N, st["weight"], EPS, st["sum"], N, None, N, st["q"], _ld(N),
                     st["scales"])
        return head + (st["q"][:, :N], st["scales"])
    g.sgemm_norm(T, N, st["x"], N, st["residual"], N, st["weight"], EPS, st["sum"], N, st["y"], N, None, N, None)
    if not c["train"]:
        return head + (st["y"],)
    h = st["x"] if st["residual"] is None else st["sum"]
    g.sgemm_norm_grad(T, N, h, N, st["weight"], EPS, st["dy"], N, st["dsum"], N, st["dh"], N, 0.0, st["dweight"],
                      _own_space(st, g.sgemm_norm_grad_workspace_size, T, N))
    return head + (st["y"], st["dh"], st["dweight"])


def _own_quantize(st, c):
    import fp32_gemm_03_amd as g
    T, N = c["T"], c["N"]
    g.sgemm_quantize(T, N, st["x"], N, _own_act(g, c["act"] or "silu"), st["gate"], N, st["q"], _ld(N), st["scales"])
    return st["q"][:, :N], st["scales"]


def _own_i8(st, c):
    import fp32_gemm_03_amd as g
    M, N, K = c["M"], c["N"], c["K"]
    g.sgemm_i8(M, N, K, 1.0, st["A"], _ld(K), st["a_scales"], st["B"], _ld(K), st["b_scales"], 0.0, st["C"], N)
    return st["C"]


def _own_gated_case(st, c):
    import fp32_gemm_03_amd as g
    T, N, K = c["T"], c["N"], c["K"]
    act = _own_act(g, c["act"])
    if not c["train"]:
        g.sgemm_gated(T, N, K, act, st["x"], K, st["G"], N, st["U"], N, st["y"], N, None, N, None, N)
        return st["y"]
    g.sgemm_gated(T, N, K, act, st["x"], K, st["G"], N, st["U"], N, st["y"], N, st["gate"], N, st["up"], N)
    g.sgemm_gated_grad(T, N, K, act, st["x"], K, st["G"], N, st["U"], N, st["gate"], N, st["up"], N, st["dy"], N,
                       st["dx"], K, 0.0, st["dG"], N, st["dU"], N,
                       _own_space(st, g.sgemm_gated_grad_workspace_size, T, N, K))
    return st["y"], st["dx"], st["dG"], st["dU"]


def _own_block(st, c):
    import fp32_gemm_03_amd as g
    T, N, K = c["T"], c["N"], c["K"]
    H = st["H"]
    g.sgemm_norm(T, K, st["x"], K, st["residual"], K, st["weight"], EPS, st["sum"], K, None, K, st["q"], _ld(K),
                 st["scales"])
    g.sgemm_i8(T, 2 * N, K, 1.0, st["q"], _ld(K), st["scales"], st["B"], _ld(K), st["b_scales"], 0.0, H, 2 * N)
    g.sgemm_quantize(T, N, H[:, N:], 2 * N, _own_act(g, c["act"]), H, 2 * N, st["q2"], _ld(N), st["scales2"])
    g.sgemm_i8(T, K, N, 1.0, st["q2"], _ld(N), st["scales2"], st["B2"], _ld(N), st["b2_scales"], 1.0, st["sum"], K)
    return st["q"][:, :K], st["scales"], st["q2"][:, :N], st["scales2"], st["sum"]


def run(st):
    c = st["case"]
    op = c["op"]
    if op == "norm":
        return _own_norm_case(st, c) if own else _plain_norm_case(st, c)
    if op == "quantize":
        if own:
            return _own_quantize(st, c)
        if not c["act"]:
            return _plain_quantize(st["x"])
        return _plain_quantize((_plain_act(st["gate"].double(), c["act"]) * st["x"].double()).to(F32))
    if op == "i8":
        if own:
            return _own_i8(st, c)
        K = c["K"]
        return st["A"][:, :K].float() @ st["B"][:, :K].float().t() * st["a_scales"].unsqueeze(1) * st["b_scales"]
    if op == "gated":
        return _own_gated_case(st, c) if own else _plain_gated_case(st, c)
    return _own_block(st, c) if own else _plain_block(st, c)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    """Each input read once and each output written once, and the operations."""
    c = case
    if c["op"] == "norm":
        e = 1.0 * c["T"] * c["N"]
        b = 4.0 * e * (3 if c["residual"] else 1) + 4.0 * c["N"]
        b += e + 4.0 * c["T"] if c["quant"] else 4.0 * e
        fl = 6.0 * e
        if c["train"]:  # dy (and dsum) read, dh and dweight written; the rows are there already
            b += 4.0 * e * (3 if c["residual"] else 2) + 4.0 * c["N"]
            fl += 10.0 * e
        return {"bytes": b, "flops": fl}
    if c["op"] == "quantize":
        e = 1.0 * c["T"] * c["N"]
        return {"bytes": (9.0 if c["act"] else 5.0) * e + 4.0 * c["T"], "flops": (8.0 if c["act"] else 3.0) * e}
    if c["op"] == "i8":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": 1.0 * (M + N) * K + 4.0 * M * N + 4.0 * (M + N), "flops": 2.0 * M * N * K}
    T, N, K = c["T"], c["N"], c["K"]
    if c["op"] == "block":
        return {"bytes": 12.0 * T * K + 3.0 * N * K + 1.0 * T * (K + N) + 8.0 * T + 8.0 * (N + K),
                "flops": 6.0 * T * N * K}
    b, fl = 4.0 * (T * K + 2 * K * N + T * N), 4.0 * T * N * K
    if c["train"]:
        b, fl = b + 4.0 * (T * N + T * K + 2 * K * N), 3 * fl
    return {"bytes": b, "flops": fl}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_act(g, act):
    f = torch.nn.functional
    return f.silu(g) if act == "silu" else f.gelu(g, approximate="tanh" if act == "gelu_tanh" else "none")


def _exact_scales(v):
    return torch.linalg.vector_norm(v, math.inf, dim=1) / 127.0


def _exact_rms(h, weight):
    return h * torch.rsqrt(h.pow(2).sum(1, keepdim=True) / h.shape[1] + EPS) * weight


def _exact_gated(st, act):
    """y and, from the graph, what the gradients of <dy, y> are."""
    x, G, U = (st[n].double().requires_grad_("dy" in st) for n in ("x", "G", "U"))
    y = _exact_act(torch.mm(x, G), act) * torch.mm(x, U)
    if "dy" not in st:
        return y
    return (y.detach(), *torch.autograd.grad(y, (x, G, U), st["dy"].double()))


def exact(case, seed):
    c, st = case, prepare(case, seed)
    op = c["op"]
    if op == "norm":
        h = st["x"].double()
        head = ()
        if c["residual"]:
            h = torch.add(h, st["residual"])
            head = (h,)
            h = h.to(F32).double()  # the sum is rounded, and what follows is of the rounded one
        w = st["weight"].double()
        if c["train"]:
            h, w = h.requires_grad_(True), w.requires_grad_(True)
        y = _exact_rms(h, w)
        if c["quant"]:
            return head + (None, _exact_scales(y))
        if not c["train"]:
            return head + (y,)
        loss = (y * st["dy"]).sum() + (0.0 if st["dsum"] is None else (h * st["dsum"]).sum())
        return head + (y.detach(), *torch.autograd.grad(loss, (h, w)))
    if op == "quantize":
        v = st["x"].double()
        if c["act"]:
            v = v * _exact_act(st["gate"].double(), c["act"])
        return None, _exact_scales(v)
    if op == "i8":
        K = c["K"]
        A = st["A"][:, :K].double()
        return torch.mm(A * st["a_scales"].double()[:, None], (st["B"][:, :K].double() * st["b_scales"].double()[:, None]).t())
    if op == "gated":
        return _exact_gated(st, c["act"])
    N, K = c["N"], c["K"]
    h = (st["x"].double() + st["residual"].double()).to(F32).double()
    y = _exact_rms(h, st["weight"].double()).to(F32).double()
    s = _exact_scales(y)
    # whole numbers of 127 y / max |y|, halves to the even one
    q = torch.round(y * (1.0 / s).unsqueeze(1))
    H = torch.mm(q * s.to(F32).double()[:, None], (st["B"][:, :K].double() * st["b_scales"].double()[:, None]).t())
    H = H.to(F32).double()
    v = (_exact_act(H[:, :N], c["act"]) * H[:, N:]).to(F32).double()
    s2 = _exact_scales(v)
    q2 = torch.round(v * (1.0 / s2).unsqueeze(1))
    B2 = st["B2"][:, :N].double() * st["b2_scales"].double()[:, None]
    return None, s, None, s2, torch.mm(q2 * s2.to(F32).double()[:, None], B2.t()) + h
