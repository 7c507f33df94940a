"""What is measured of the row-wise products: the router, the experts' products and the
low-rank adapters, each with its gradients.

Every case names an operator (``op``) and its sizes:

* ``route``    -- router scores -> the experts of each token and their weights, and back;
* ``experts``  -- rows grouped by expert, the experts' products, the weighted sum per token;
                  ``train`` adds the gradients of the tokens, the experts and the weights;
* ``adapters`` -- a shared projection with a low-rank adapter per row; ``train`` adds the
                  gradients of the rows and of the adapters;
* ``layer``    -- the router and two experts' products with an activation between them.

``run`` computes the plain form (elementary torch operations; sums in 32 bits, the router in
64) or, where ``own`` is true, calls the library.
"""
import math

import torch

own = False

F32 = torch.float32
SOFTMAX, SIGMOID = 0, 1


def listed():
    return [
        # one sequence being decoded: latency is all there is
        {"name": "route one token", "op": "route", "T": 1, "E": 64, "k": 4, "sigmoid": False, "bias": False,
         "groups": 1, "top_groups": 1, "best": 1, "renorm": True, "scale": 1.0, "ties": False, "train": False},
        # a prompt through a router with a bias for balance and groups of experts; odd length
        {"name": "route sigmoid groups", "op": "route", "T": 8191, "E": 256, "k": 8, "sigmoid": True, "bias": True,
         "groups": 8, "top_groups": 4, "best": 2, "renorm": True, "scale": 2.5, "ties": False, "train": False},
        # a training batch: scores that came from 16 bits (ties), weights not renormalised, and back
        {"name": "route train", "op": "route", "T": 16384, "E": 64, "k": 6, "sigmoid": False, "bias": False,
         "groups": 1, "top_groups": 1, "best": 1, "renorm": False, "scale": 1.0, "ties": True, "train": True},
        # one token through its experts: the experts' weights are read once
        {"name": "experts one token", "op": "experts", "T": 1, "E": 16, "k": 2, "K": 2048, "N": 1024,
         "trans": False, "pad": 0, "train": False},
        # a batch of sequences being decoded, experts stored output-major, ragged rows per expert
        {"name": "experts decode batch", "op": "experts", "T": 37, "E": 64, "k": 4, "K": 2048, "N": 1280,
         "trans": True, "pad": 3, "train": False},
        # a long prompt: matrix-product bound
        {"name": "experts prompt", "op": "experts", "T": 4096, "E": 16, "k": 2, "K": 2048, "N": 4096,
         "trans": False, "pad": 0, "train": False},
        # a training step of odd length with padded tokens
        {"name": "experts train", "op": "experts", "T": 2011, "E": 8, "k": 2, "K": 1024, "N": 2048,
         "trans": True, "pad": 50, "train": True},
        # one sequence with an adapter being decoded
        {"name": "adapters one token", "op": "adapters", "M": 1, "N": 4096, "K": 4096, "G": 8, "rank": 16,
         "requests": 1, "train": False},
        # a batch of sequences, each with its own adapter, of several ranks
        {"name": "adapters decode batch", "op": "adapters", "M": 29, "N": 4095, "K": 2048, "G": 32, "rank": 64,
         "requests": 29, "train": False},
        # several prompts in one batch, each with its own adapter
        {"name": "adapters prompts", "op": "adapters", "M": 4096, "N": 4096, "K": 2048, "G": 16, "rank": 32,
         "requests": 11, "train": False},
        # a training step over sequences of several adapters
        {"name": "adapters train", "op": "adapters", "M": 2000, "N": 2048, "K": 1024, "G": 6, "rank": 16,
         "requests": 9, "train": True},
        # the router and the experts together, as a model's layer runs them
        {"name": "expert layer", "op": "layer", "T": 515, "E": 32, "k": 4, "K": 1024, "N": 1408,
         "sigmoid": True, "bias": True, "groups": 4, "top_groups": 2, "best": 2, "renorm": True, "scale": 1.0,
         "ties": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the ranges above: token counts, widths and expert counts spread over
    their logarithm and mostly odd, every option drawn, work below the largest listed case's."""
    op = rng.choice(["route", "experts", "adapters", "layer"])
    if op in ("route", "layer"):
        e_log = rng.randint(3, 8 if op == "route" else 6)
        groups = rng.choice([1, 1, 2, 4])
        e = groups * max(2, (1 << e_log) // groups + rng.choice([-1, 0, 0, 1]))
        top_groups = rng.randint(1, groups)
        k = min(rng.choice([1, 2, 3, 4, 6, 8]), e // groups * top_groups)
        score = {"sigmoid": rng.random() < 0.5, "bias": rng.random() < 0.5, "groups": groups,
                 "top_groups": top_groups, "best": rng.choice([1, 2]), "renorm": rng.random() < 0.5,
                 "scale": rng.choice([1.0, 2.5]), "ties": rng.random() < 0.5}
        if op == "route":
            return {"op": op, "T": _log(rng, 1, 16384), "E": e, "k": k, **score, "train": rng.random() < 0.5}
        return {"op": op, "T": _log(rng, 1, 1024), "E": e, "k": k, "K": _log(rng, 100, 1024),
                "N": _log(rng, 100, 1500), **score}
    train = rng.random() < 0.4
    if op == "experts":
        e = rng.choice([4, 7, 8, 16, 32, 60])
        k = rng.choice([1, 2, 3, 4])
        t = _log(rng, 1, 2048 if train else 4096)
        kk, n = _log(rng, 128, 2048), _log(rng, 128, 2048)
        while e * kk * n > 1 << 27 or t * k * kk * n > 1 << (34 if train else 35):
            kk, n = (kk * 3 // 4, n) if kk > n else (kk, n * 3 // 4)
        return {"op": op, "T": t, "E": e, "k": k, "K": kk, "N": n, "trans": rng.random() < 0.5,
                "pad": rng.choice([0, t // 7]), "train": train}
    m = _log(rng, 1, 2048 if train else 4096)
    n, kk = _log(rng, 256, 4096), _log(rng, 256, 4096)
    while m * n * kk > 1 << (32 if train else 35):
        n, kk = (n * 3 // 4, kk) if n > kk else (n, kk * 3 // 4)
    return {"op": op, "M": m, "N": n, "K": kk, "G": _log(rng, 1, 32), "rank": rng.choice([4, 8, 16, 24, 32, 64]),
            "requests": min(m, _log(rng, 1, 48)), "train": train}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _scores(gen, case, dev):
    """Router scores: a spread of 1.5 as trained routers have, 2% of them masked, the last
    twentieth of the tokens padding (every score masked), and the bias that balances."""
    T, E = case["T"], case["E"]
    logits = torch.randn(T, E, generator=gen, device=dev) * 1.5
    if case["ties"]:
        logits = logits.to(torch.bfloat16).to(F32)
    logits.masked_fill_(torch.rand(T, E, generator=gen, device=dev) < 0.02, -math.inf)
    if T >= 20:
        logits[T - T // 20:] = -math.inf
    bias = torch.randn(E, generator=gen, device=dev) * 0.1 if case["bias"] else None
    return logits, bias


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(1000003 * int(seed) + 17)
    rnd = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    empty = lambda *s: torch.empty(*s, dtype=F32, device=dev)  # noqa: E731
    ints = lambda *s: torch.full(s, -1, dtype=torch.int32, device=dev)  # noqa: E731
    st = {"case": case}
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        st["logits"], st["bias"] = _scores(gen, case, dev)
        st["ids"], st["weights"] = ints(T, k), empty(T, k)
        if case["train"]:
            st["dweights"], st["dlogits"] = rnd(T, k), empty(T, E)
        return st
    if case["op"] == "experts":
        T, E, k, K, N = (case[n] for n in ("T", "E", "k", "K", "N"))
        R = T * k
        popular = rnd(E) * 0.3
        st["ids"] = torch.topk(rnd(T, E) + popular, k, dim=1).indices.to(torch.int32).contiguous()
        if case["pad"]:
            st["ids"][T - case["pad"]:] = -1
        st["weights"] = torch.softmax(rnd(T, k), 1).contiguous()
        st["x"] = rnd(T, K)
        st["B"] = (rnd(E, N, K) if case["trans"] else rnd(E, K, N)) / math.sqrt(K)
        st["offsets"], st["rows"] = ints(E + 1), ints(R)
        st["Y"], st["out"] = empty(R, N), empty(T, N)
        if case["train"]:
            st["dout"], st["dY"], st["dweights"] = rnd(T, N), empty(R, N), empty(T, k)
            st["dA"], st["dx"], st["dB"] = empty(R, K), empty(T, K), torch.empty_like(st["B"])
        return st
    if case["op"] == "adapters":
        M, N, K, G, r = (case[n] for n in ("M", "N", "K", "G", "rank"))
        # requests of uneven lengths, one after the other; about a tenth has no adapter
        cuts = torch.sort(torch.rand(M, generator=gen, device=dev)).values
        request = (cuts * case["requests"]).long().clamp_(max=case["requests"] - 1)
        if case["requests"] == M:
            request = torch.arange(M, device=dev)
        of_request = torch.randint(0, G, (case["requests"],), generator=gen, device=dev)
        if case["requests"] > 1:
            none = torch.rand(case["requests"], generator=gen, device=dev) < 0.1
            of_request = torch.where(none, -1, of_request)
        st["ids"] = of_request[request].to(torch.int32).contiguous()
        st["ranks"] = torch.randint(max(1, r // 4), r + 1, (G,), generator=gen, device=dev).to(torch.int32)
        st["scales"] = 0.5 + torch.rand(G, generator=gen, device=dev)
        st["A"], st["B"] = rnd(M, K), rnd(K, N) / math.sqrt(K)
        st["U"], st["V"] = rnd(G, K, r) / math.sqrt(K), rnd(G, r, N) / math.sqrt(r)
        st["C"] = empty(M, N)
        if case["train"]:
            st["dC"], st["dA"] = rnd(M, N), empty(M, K)
            st["dU"], st["dV"] = torch.empty_like(st["U"]), torch.empty_like(st["V"])
        return st
    T, E, k, K, N = (case[n] for n in ("T", "E", "k", "K", "N"))
    R = T * k
    st["logits"], st["bias"] = _scores(gen, case, dev)
    st["x"] = rnd(T, K)
    st["B"], st["B2"] = rnd(E, K, N) / math.sqrt(K), rnd(E, N, K) / math.sqrt(N)
    st["ids"], st["weights"] = ints(T, k), empty(T, k)
    st["offsets"], st["rows"] = ints(E + 1), ints(R)
    st["H"], st["Y"], st["out"] = empty(R, N), empty(R, K), empty(T, K)
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _plain_route(logits, bias, c):
    E, k, G = c["E"], c["k"], c["groups"]
    x = logits.double()
    live = x > -math.inf
    if c["sigmoid"]:
        s = 1.0 / (1.0 + torch.exp(-x))
    else:
        top = x.max(1, keepdim=True).values
        e = torch.exp(x - torch.where(top > -math.inf, top, torch.zeros_like(top)))
        total = e.sum(1, keepdim=True)
        s = torch.where(total > 0, e / total, torch.zeros_like(e))
    # without a bias and a sum of scores, the scores' order is that of the logits
    key = x if bias is None and c["best"] == 1 else s if bias is None else s + bias.double()
    key = torch.where(live, key, torch.full_like(key, -math.inf))
    if G > 1:
        in_group = torch.sort(key.view(-1, G, E // G), dim=2, descending=True).values[:, :, :c["best"]]
        has = in_group[:, :, 0] > -math.inf
        of_group = torch.where(in_group > -math.inf, in_group, torch.zeros_like(in_group)).sum(2)
        of_group = torch.where(has, of_group, torch.full_like(of_group, -math.inf))
        order = torch.sort(of_group, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        kept = torch.zeros_like(has).scatter_(1, order, True).repeat_interleave(E // G, 1)
        key = torch.where(kept, key, torch.full_like(key, -math.inf))
    best, ids = torch.sort(key, dim=1, descending=True, stable=True)
    best, ids = best[:, :k], ids[:, :k]
    found = best > -math.inf
    w = torch.where(found, s.gather(1, ids), torch.zeros_like(best))
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return torch.where(found, ids, -1).to(torch.int32), (w * c["scale"]).to(F32), s


def _plain_route_grad(s, ids, dweights, c):
    found = ids >= 0
    at = ids.long().clamp(min=0)
    picked = torch.where(found, s.gather(1, at), torch.zeros_like(dweights, dtype=s.dtype))
    d = torch.where(found, dweights.double() * c["scale"], torch.zeros_like(picked))
    if c["renorm"]:
        total = picked.sum(1, keepdim=True)
        inv = torch.where(total > 0, 1.0 / total, torch.zeros_like(total))
        d = (d - (d * picked).sum(1, keepdim=True) * inv) * inv
    d = torch.where(found, d, torch.zeros_like(d))
    ds = torch.zeros_like(s).scatter_add_(1, at, d)
    if c["sigmoid"]:
        return (ds * s * (1.0 - s)).to(F32)
    return (s * (ds - (ds * s).sum(1, keepdim=True))).to(F32)


def _plain_groups(ids, E):
    """The flat slots sorted by expert (stable), where each expert's begin, and each slot's
    place in a table of one row of slots per expert."""
    flat = ids.reshape(-1).long()
    flat = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E + 1)
    begin = torch.cumsum(counts, 0) - counts
    offsets = begin.to(torch.int32)
    placed = torch.arange(flat.numel(), device=flat.device) < begin[E]
    rows = torch.where(placed, order, -1).to(torch.int32)
    most = int(counts[:E].max())
    here = order[:int(begin[E])]
    place = flat[here] * most + torch.arange(here.numel(), device=flat.device) - begin[flat[here]]
    return offsets, rows, most, here, place


def _padded(src, place, E, most):
    table = torch.zeros(E * most, src.shape[1], dtype=src.dtype, device=src.device)
    table[place] = src
    return table.view(E, most, -1)


def _plain_products(x, B, trans, ids, groups, E, div):
    """Row ids[slot] of every slot's product; few slots take their own copy of the weights,
    many are laid out in one padded batch."""
    _, _, most, here, place = groups
    R, N = ids.numel(), B.shape[1] if trans else B.shape[2]
    y = torch.zeros(R, N, device=x.device)
    if here.numel() == 0:
        return y
    if here.numel() <= E // 2:
        w = B[ids.reshape(-1)[here].long()]
        a = x[here // div].unsqueeze(1)
        y[here] = torch.bmm(a, w.transpose(1, 2) if trans else w).squeeze(1)
        return y
    a = _padded(x[here // div], place, E, most)
    y[here] = torch.bmm(a, B.transpose(1, 2) if trans else B).view(E * most, N)[place]
    return y


def _plain_experts(st, c):
    T, E, k = c["T"], c["E"], c["k"]
    ids, w = st["ids"], st["weights"]
    groups = _plain_groups(ids, E)
    y = _plain_products(st["x"], st["B"], c["trans"], ids, groups, E, k)
    used = torch.where(ids >= 0, w, torch.zeros_like(w))
    out = (y.view(T, k, -1) * used.unsqueeze(2)).sum(1)
    if not c["train"]:
        return groups[0], groups[1], out
    _, _, most, here, place = groups
    dy = (st["dout"].unsqueeze(1) * used.unsqueeze(2)).view(T * k, -1)
    dw = torch.where(ids >= 0, (y.view(T, k, -1) * st["dout"].unsqueeze(1)).sum(2), torch.zeros_like(w))
    dyp = _padded(dy[here], place, E, most)
    xp = _padded(st["x"][here // k], place, E, most)
    dxs = torch.zeros(T * k, c["K"], device=dy.device)
    dxs[here] = torch.bmm(dyp, st["B"] if c["trans"] else st["B"].transpose(1, 2)).view(E * most, -1)[place]
    dx = dxs.view(T, k, -1).sum(1)
    dB = torch.bmm(dyp.transpose(1, 2), xp) if c["trans"] else torch.bmm(xp.transpose(1, 2), dyp)
    return groups[0], groups[1], out, dx, dB, dw


def _plain_adapters(st, c):
    """Rows laid out in one padded batch per adapter; ranks below the largest are masked."""
    G, r = c["G"], c["rank"]
    A, B, ids = st["A"], st["B"], st["ids"]
    out = A @ B
    _, _, most, here, place = _plain_groups(ids, G)
    keep = torch.arange(r, device=A.device) < st["ranks"].unsqueeze(1)
    U = st["U"] * keep.unsqueeze(1)
    V = st["V"] * keep.unsqueeze(2)
    s = st["scales"].view(G, 1, 1)
    some = here.numel() > 0
    if some:
        a = _padded(A[here], place, G, most)
        h = torch.bmm(a, U) * s
        out[here] += torch.bmm(h, V).view(G * most, -1)[place]
    if not c["train"]:
        return out
    dC = st["dC"]
    dA = dC @ B.t()
    dU, dV = torch.zeros_like(U), torch.zeros_like(V)
    if some:
        d = _padded(dC[here], place, G, most)
        dh = torch.bmm(d, V.transpose(1, 2)) * s
        dA[here] += torch.bmm(dh, U.transpose(1, 2)).view(G * most, -1)[place]
        dU = torch.bmm(a.transpose(1, 2), dh)
        dV = torch.bmm(h.transpose(1, 2), d)
    return out, dA, dU, dV


def _plain_layer(st, c):
    ids, w, _ = _plain_route(st["logits"], st["bias"], c)
    E, k = c["E"], c["k"]
    groups = _plain_groups(ids, E)
    h = _plain_products(st["x"], st["B"], False, ids, groups, E, k)
    h = h / (1.0 + torch.exp(-h))
    y = _plain_products(h, st["B2"], False, ids, groups, E, 1)
    out = (y.view(c["T"], k, -1) * w.unsqueeze(2)).sum(1)
    return ids, w, out


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own_route(st, c):
    import fp32_gemm_03_amd as g
    g.sgemm_route(c["T"], c["E"], c["k"], SIGMOID if c["sigmoid"] else SOFTMAX, st["logits"], c["E"], st["bias"],
                  c["groups"], c["top_groups"], c["best"], c["renorm"], c["scale"], st["ids"], st["weights"])


def _own_space(st, size, *args):
    if "space" not in st:  # a program keeps its workspace
        st["space"] = torch.empty(max(256, size(*args)), dtype=torch.uint8, device="cuda")
    return st["space"]


def _own_group(st, R, G):
    import fp32_gemm_03_amd as g
    g.sgemm_group_rows(R, G, st["ids"], st["offsets"], st["rows"],
                       _own_space(st, g.sgemm_group_rows_workspace_size, R, G))


def _own_experts(st, c):
    import fp32_gemm_03_amd as g
    T, E, k, K, N = (c[n] for n in ("T", "E", "k", "K", "N"))
    R, ldb = T * k, K if c["trans"] else N
    _own_group(st, R, E)
    g.sgemm_grouped(E, R, N, K, 1.0, st["x"], K, k, st["B"], ldb, K * N, c["trans"], 0.0, st["Y"], N, True,
                    st["offsets"], st["rows"])
    g.sgemm_combine(T, k, N, E, st["ids"], st["weights"], st["Y"], N, 0.0, st["out"], N)
    if not c["train"]:
        return st["offsets"], st["rows"], st["out"]
    g.sgemm_combine_grad(T, k, N, E, st["ids"], st["weights"], st["dout"], N, st["Y"], N, st["dY"], N,
                         st["dweights"])
    g.sgemm_grouped(E, R, K, N, 1.0, st["dY"], N, 1, st["B"], ldb, K * N, not c["trans"], 0.0, st["dA"], K, True,
                    st["offsets"], st["rows"])
    g.sgemm_combine(T, k, K, E, st["ids"], None, st["dA"], K, 0.0, st["dx"], K)
    if c["trans"]:
        g.sgemm_grouped_tn(E, R, N, K, 1.0, st["dY"], N, 1, st["x"], K, k, 0.0, st["dB"], K, K * N,
                           st["offsets"], st["rows"])
    else:
        g.sgemm_grouped_tn(E, R, K, N, 1.0, st["x"], K, k, st["dY"], N, 1, 0.0, st["dB"], N, K * N,
                           st["offsets"], st["rows"])
    return st["offsets"], st["rows"], st["out"], st["dx"], st["dB"], st["dweights"]


def _own_adapters(st, c):
    import fp32_gemm_03_amd as g
    M, N, K, G, r = (c[n] for n in ("M", "N", "K", "G", "rank"))
    size = g.sgemm_adapters_grad_workspace_size if c["train"] else g.sgemm_adapters_workspace_size
    space = _own_space(st, size, M, N, K, G, r)
    g.sgemm_adapters(M, N, K, 1.0, st["A"], K, st["B"], N, 0.0, st["C"], N, G, r, st["ids"], st["ranks"],
                     st["scales"], st["U"], r, K * r, st["V"], N, r * N, space)
    if not c["train"]:
        return st["C"]
    g.sgemm_adapters_grad(M, N, K, 1.0, st["A"], K, st["B"], N, st["dC"], N, G, r, st["ids"], st["ranks"],
                          st["scales"], st["U"], r, K * r, st["V"], N, r * N, 0.0, st["dA"], K, st["dU"], r, K * r,
                          st["dV"], N, r * N, space)
    return st["C"], st["dA"], st["dU"], st["dV"]


def _own_layer(st, c):
    import fp32_gemm_03_amd as g
    T, E, k, K, N = (c[n] for n in ("T", "E", "k", "K", "N"))
    R = T * k
    _own_route(st, c)
    _own_group(st, R, E)
    g.sgemm_grouped(E, R, N, K, 1.0, st["x"], K, k, st["B"], N, K * N, False, 0.0, st["H"], N, False,
                    st["offsets"], st["rows"])
    h = torch.nn.functional.silu(st["H"])
    g.sgemm_grouped(E, R, K, N, 1.0, h, N, 0, st["B2"], K, K * N, False, 0.0, st["Y"], K, True,
                    st["offsets"], st["rows"])
    g.sgemm_combine(T, k, K, E, st["ids"], st["weights"], st["Y"], K, 0.0, st["out"], K)
    return st["ids"], st["weights"], st["out"]


def run(st):
    c = st["case"]
    op = c["op"]
    if op == "route":
        if own:
            import fp32_gemm_03_amd as g
            _own_route(st, c)
            if not c["train"]:
                return st["ids"], st["weights"]
            g.sgemm_route_grad(c["T"], c["E"], c["k"], SIGMOID if c["sigmoid"] else SOFTMAX, st["logits"], c["E"],
                               c["renorm"], c["scale"], st["ids"], st["dweights"], st["dlogits"], c["E"])
            return st["ids"], st["weights"], st["dlogits"]
        ids, weights, s = _plain_route(st["logits"], st["bias"], c)
        if not c["train"]:
            return ids, weights
        return ids, weights, _plain_route_grad(s, ids, st["dweights"], c)
    if op == "experts":
        return _own_experts(st, c) if own else _plain_experts(st, c)
    if op == "adapters":
        return _own_adapters(st, c) if own else _plain_adapters(st, c)
    return _own_layer(st, c) if own else _plain_layer(st, c)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _active(groups, rows):
    """Groups that hold at least one of so many rows spread evenly."""
    return groups * (1.0 - (1.0 - 1.0 / groups) ** rows)


def work(case):
    """Each input read once and each output written once (experts and adapters that no row
    uses are not read), and the products' operations."""
    c = case
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        b = 4.0 * T * E + 8.0 * T * k + (4.0 * E if c["bias"] else 0.0)
        fl = 6.0 * T * E
        if c["train"]:
            b, fl = b + 4.0 * T * E + 4.0 * T * k, fl * 2
        return {"bytes": b, "flops": fl}
    if c["op"] == "adapters":
        M, N, K, G, r = (c[n] for n in ("M", "N", "K", "G", "rank"))
        g, r = _active(G, c["requests"]), 0.625 * r
        b = 4.0 * (M * K + K * N + M * N + g * r * (K + N)) + 4.0 * M
        fl = 2.0 * M * (K * N + r * (K + N))
        if c["train"]:  # dC read once, dA, dU and dV written; dU and dV whole
            b += 4.0 * (M * N + M * K + G * c["rank"] * (K + N))
            fl += 2.0 * M * (K * N + 3 * r * (K + N))
        return {"bytes": b, "flops": fl}
    T, E, k, K, N = (c[n] for n in ("T", "E", "k", "K", "N"))
    rows = (T - c.get("pad", 0)) * k if c["op"] == "experts" else (T - T // 20) * k if T >= 20 else T * k
    e = _active(E, rows)
    if c["op"] == "layer":
        return {"bytes": 4.0 * (2 * T * K + 2 * e * K * N + T * E) + 8.0 * T * k, "flops": 4.0 * rows * K * N}
    b = 4.0 * (T * K + e * K * N + T * N) + 12.0 * T * k
    fl = 2.0 * rows * (K + 1) * N
    if c["train"]:
        b, fl = b + 4.0 * (T * N + T * K + E * K * N) + 4.0 * T * k, 3 * fl
    return {"bytes": b, "flops": fl}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_route(logits, bias, c):
    """Row by row on the host, from the definition; returns ids and, differentiable, weights."""
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    x = logits.double().cpu().requires_grad_(True)
    if c["sigmoid"]:
        score = torch.sigmoid(x)
    else:
        score = torch.softmax(x.where((x > -math.inf).any(1, keepdim=True), torch.zeros(1, dtype=x.dtype)), 1)
    xs, ss = x.detach().numpy(), score.detach().numpy()
    b = None if bias is None else bias.double().cpu().numpy()
    logit_order = b is None and c["best"] == 1
    picks = []
    for t in range(T):
        key = [xs[t, e] if logit_order else ss[t, e] + (0.0 if b is None else b[e]) for e in range(E)]
        cand = [e for e in range(E) if xs[t, e] > -math.inf]
        if G > 1:
            per = E // G
            value = {}
            for e in cand:
                value.setdefault(e // per, []).append(key[e])
            value = {g: sum(sorted(v, reverse=True)[:c["best"]]) for g, v in value.items()}
            kept = set(sorted(value, key=lambda g: (-value[g], g))[:c["top_groups"]])
            cand = [e for e in cand if e // per in kept]
        cand.sort(key=lambda e: (-key[e], e))
        picks.append(cand[:k] + [-1] * (k - len(cand[:k])))
    ids = torch.tensor(picks, dtype=torch.int32).view(T, k)
    w = score.gather(1, ids.long().clamp(min=0)) * (ids >= 0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / total.where(total > 0, torch.ones(1, dtype=w.dtype))
    return x, ids, w * c["scale"]


def _exact_products(x, B, trans, ids, weights):
    """sum_j weights[t, j] x[t] B[ids[t, j]], one expert at a time."""
    out = None
    for e in range(B.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        y = x[t] @ (B[e].t() if trans else B[e])
        part = torch.zeros(x.shape[0], y.shape[1], dtype=y.dtype, device=y.device)
        part = part.index_add(0, t, y * weights[t, j].unsqueeze(1))
        out = part if out is None else out + part
    return out


def exact(case, seed):
    st, c = prepare(case, seed), case
    if c["op"] == "route":
        x, ids, w = _exact_route(st["logits"], st["bias"], c)
        if not c["train"]:
            return ids, w.detach()
        w.backward(st["dweights"].double().cpu())
        # a masked expert's score does not depend on its logit; its gradient is 0
        return ids, w.detach(), torch.nan_to_num(x.grad, nan=0.0)
    if c["op"] == "layer":
        _, ids, w = _exact_route(st["logits"], st["bias"], c)
        ids, w = ids.cuda(), w.detach().cuda()
        x, b1, b2 = st["x"].double(), st["B"].double(), st["B2"].double()
        out = torch.zeros_like(x)
        for e in range(c["E"]):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            h = x[t] @ b1[e]
            out.index_add_(0, t, ((h * torch.sigmoid(h)) @ b2[e]) * w[t, j].unsqueeze(1))
        return ids, w, out
    if c["op"] == "experts":
        flat = st["ids"].reshape(-1).cpu().tolist()
        lists = [[i for i, v in enumerate(flat) if v == e] for e in range(c["E"])]
        starts = [0]
        for v in lists:
            starts.append(starts[-1] + len(v))
        rows = [i for v in lists for i in v]
        rows += [-1] * (len(flat) - len(rows))
        heads = (torch.tensor(starts, dtype=torch.int32), torch.tensor(rows, dtype=torch.int32))
        x, B, w = (st[n].double().requires_grad_(c["train"]) for n in ("x", "B", "weights"))
        out = _exact_products(x, B, c["trans"], st["ids"], w)
        if not c["train"]:
            return (*heads, out)
        out.backward(st["dout"].double())
        return (*heads, out.detach(), x.grad, B.grad, w.grad)
    A, B, U, V = (st[n].double() for n in ("A", "B", "U", "V"))
    if c["train"]:
        A, U, V = (v.requires_grad_(True) for v in (A, U, V))
    out = A @ B
    for a in range(c["G"]):
        rows = torch.nonzero(st["ids"] == a).reshape(-1)
        n = int(st["ranks"][a])
        d = (A[rows] @ U[a, :, :n]) @ V[a, :n] * st["scales"][a].double()
        out = out.index_add(0, rows, d)
    if not c["train"]:
        return out
    out.backward(st["dC"].double())
    return out.detach(), A.grad, U.grad, V.grad
