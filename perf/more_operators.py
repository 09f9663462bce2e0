"""The Muon operators: what is measured of them, and their plain forms.

The update of weight matrices by their orthogonalised momentum, next to AdamW:

  orth   a stack of matrices of one shape, orthogonalised by Newton-Schulz steps: X = G / (|G| + eps) with the
         Frobenius norm, then per step (a, b, c): A = X X^T on the smaller side, X = a X + (b A + c A^2) X;
         bf16 or fp32 in, bf16 out
  stack  the whole update of a stack of matrices of one shape: with g = grad * clip, momentum = mu * momentum + g,
         u = g + mu * momentum (or the momentum itself), O = orth(u) in bf16,
         master = master * (1 - lr * wd) - (lr * scale) * O, param = bf16(master)
  list   the same over a list of matrices of any shapes, described once in a table

The plain forms are elementary torch operations in fp32. `exact` states the same operators in 64 bits (and does not
round the orthogonalised update, which zero_orthogonalize returns and the updates use in bf16).
"""
import math

import torch

own = False

STEPS = [(3.4445, -4.7750, 2.0315)] * 5
EPS = 1e-7
LR, MU, WD = 4e-4, 0.95, 0.1


# ----------------------------------------------------------------- the cases

def listed():
    return [
        # the 12 heads' rows of one GPT-2-small attention projection, each head on its own: latency
        {"name": "orth 12 x 64x768 bf16", "op": "orth", "count": 12, "rows": 64, "cols": 768, "fp32": False},
        # the odd matrix of a 1 M-parameter model
        {"name": "orth 487x1000 fp32", "op": "orth", "count": 1, "rows": 487, "cols": 1000, "fp32": True},
        # GPT-2 small's attention output projections, all layers at once
        {"name": "orth 12 x 768x768 bf16", "op": "orth", "count": 12, "rows": 768, "cols": 768, "fp32": False},
        # Llama-3-8B's MLP gate (tall)
        {"name": "orth 14336x4096 bf16", "op": "orth", "count": 1, "rows": 14336, "cols": 4096, "fp32": False},
        # one rank's share of GPT-2 small's attention projections, stacked
        {"name": "stack 2 x 768x2304", "op": "stack", "count": 2, "rows": 768, "cols": 2304},
        # Llama-3-70B's attention projection, two layers
        {"name": "stack 2 x 8192x8192", "op": "stack", "count": 2, "rows": 8192, "cols": 8192},
        # the 1 M-parameter model's matrices
        {"name": "list tiny 2", "op": "list", "kind": "tiny"},
        # one rank of 8 of GPT-2 small: 6 of its 48 matrices
        {"name": "list gpt 6", "op": "list", "kind": "gpt", "d": 768, "matrices": 6},
        # many small odd matrices: adapters, routers, projections of small models
        {"name": "list ragged 40", "op": "list", "kind": "ragged", "matrices": 40, "least": 8, "most": 600, "shape_seed": 3},
        # one rank of 8 of a 1.3 B GPT: 12 of its 96 matrices
        {"name": "list gpt 12", "op": "list", "kind": "gpt", "d": 2048, "matrices": 12},
        # one layer of Llama-3-8B: seven matrices of three shapes
        {"name": "list llama 7", "op": "list", "kind": "llama", "d": 4096, "kv": 1024, "ffn": 14336},
        # Llama-3-70B's MLP matrix
        {"name": "list 8192x28672", "op": "list", "kind": "one", "rows": 8192, "cols": 28672},
    ]


def draw(rng):
    """Shapes from a few rows to thousands, spread over their logarithm, odd ones among them, wide, tall and square;
    no more work than the largest listed."""
    spread = lambda lo, hi: int(math.exp(rng.uniform(math.log(lo), math.log(hi))))  # noqa: E731
    op = rng.choice(["orth", "stack", "list"])
    if op == "list":
        least = rng.choice([4, 64])
        return {"op": op, "kind": "ragged", "matrices": spread(1, 60), "least": least, "most": spread(300, 3000),
                "shape_seed": rng.randrange(1 << 20), "nesterov": rng.random() < 0.7}
    rows = spread(8, 5000)
    cols = rows if rng.random() < 0.25 else spread(8, 12000)
    if rng.random() < 0.3:
        rows, cols = -(-rows // 64) * 64, -(-cols // 64) * 64
    count = min(spread(1, 24), max(1, 100_000_000 // (rows * cols)))
    if op == "orth":
        return {"op": op, "count": count, "rows": rows, "cols": cols, "fp32": rng.random() < 0.5}
    return {"op": op, "count": count, "rows": rows, "cols": cols, "nesterov": rng.random() < 0.7}


def _shapes(case):
    """(rows, cols) of each matrix of a case."""
    kind = case.get("kind")
    if case["op"] != "list":
        return [(case["rows"], case["cols"])] * case["count"]
    if kind == "one":
        return [(case["rows"], case["cols"])]
    if kind == "tiny":
        return [(1000, 512), (487, 1000)]
    if kind == "gpt":
        d = case["d"]
        return ([(d, 3 * d), (d, d), (d, 4 * d), (4 * d, d)] * case["matrices"])[:case["matrices"]]
    if kind == "llama":
        d, kv, ffn = case["d"], case["kv"], case["ffn"]
        return [(d, d), (kv, d), (kv, d), (d, d), (ffn, d), (ffn, d), (d, ffn)]
    gen = torch.Generator().manual_seed(case["shape_seed"])
    lo, hi = math.log(case["least"]), math.log(case["most"])
    sides = torch.exp(lo + (hi - lo) * torch.rand(case["matrices"], 2, generator=gen, dtype=torch.float64))
    return [(int(r), int(c)) for r, c in sides.tolist()]


def work(case):
    """Products of two symmetric factors that commute are symmetric: half of them is computed. Two steps can be taken
    as one on the smaller side (m^3 products in place of m^2 n ones), which is less where n > m."""
    flops = byts = 0
    for rows, cols in _shapes(case):
        m, n = min(rows, cols), max(rows, cols)
        flops += min(15 * m * m * n + 5 * m ** 3, 9 * m * m * n + 11 * m ** 3)
        byts += rows * cols * ((6 if case["fp32"] else 4) if case["op"] == "orth" else 20)
    return {"bytes": byts, "flops": flops}


# ----------------------------------------------------------------- inputs

def _spans(shapes):
    at, spans = 0, []
    for rows, cols in shapes:
        spans.append((at, rows, cols))
        at += rows * cols
    return spans, at


def prepare(case, seed):
    """Gradients as training has them: a few strong directions over noise."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, device=dev, generator=gen)  # noqa: E731
    spans, total = _spans(_shapes(case))

    def like_gradients(size):
        x = normal(total)
        for at, rows, cols in spans:
            k = min(rows, cols, 8)
            strong = normal(rows, k) * torch.exp2(-torch.arange(k, device=dev) / 2)
            x[at:at + rows * cols] += 0.5 * (strong @ normal(k, cols)).view(-1)
        return x * size

    if case["op"] == "orth":
        x = like_gradients(1e-3)
        s = {"case": case, "x": x if case["fp32"] else x.bfloat16()}
        if own:
            import zero_partitioned_mixed_partition_amd as zm
            s["out"] = torch.empty(total, dtype=torch.bfloat16, device=dev)
            s["workspace"] = zm.muon_workspace(case["count"], case["rows"], case["cols"], dev)
        return s
    grad = like_gradients(1e-3)
    s = {"case": case, "momentum": like_gradients(5e-3) + 3 * grad, "grad": grad.bfloat16(), "master": normal(total) * 0.02,
         "param": torch.zeros(total, dtype=torch.bfloat16, device=dev), "clip": torch.full((1,), 0.8125, device=dev)}
    if own:
        import zero_partitioned_mixed_partition_amd as zm
        if case["op"] == "stack":
            s["workspace"] = zm.muon_workspace(case["count"], case["rows"], case["cols"], dev)
        else:
            cut = lambda t: [t[at:at + rows * cols] for at, rows, cols in spans]  # noqa: E731
            s["table"] = zm.MuonTable(cut(s["master"]), cut(s["momentum"]), cut(s["grad"]), cut(s["param"]), _shapes(case))
    return s


# ----------------------------------------------------------------- one pass

def _plain_orth(x):
    """fp32 [count, rows, cols] orthogonalised, in bf16."""
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2).contiguous() if tall else x
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    for a, b, c in STEPS:
        gram = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.bmm(b * gram + c * torch.bmm(gram, gram), x)
    return (x.transpose(1, 2) if tall else x).bfloat16()


def _scale(rows, cols):
    """The usual factor, which gives the update the root mean square of an AdamW step."""
    return 0.2 * math.sqrt(max(rows, cols))


def run(s):
    case = s["case"]
    nesterov = case.get("nesterov", True)
    if own:
        import zero_partitioned_mixed_partition_amd as zm
        if case["op"] == "orth":
            zm.zero_orthogonalize(s["x"], s["out"], case["rows"], case["cols"], coefficients=STEPS, eps=EPS,
                                  workspace=s["workspace"])
            return s["out"]
        hyper = dict(lr=LR, momentum=MU, nesterov=nesterov, weight_decay=WD, coefficients=STEPS, eps=EPS,
                     clip_scale=s["clip"])
        if case["op"] == "stack":
            zm.zero_muon_step(s["master"], s["momentum"], s["grad"], s["param"], case["rows"], case["cols"],
                              workspace=s["workspace"], **hyper)
        else:
            s["table"].step(**hyper)
        return {k: s[k] for k in ("master", "momentum", "param")}
    if case["op"] == "orth":
        return _plain_orth(s["x"].float().view(case["count"], case["rows"], case["cols"])).reshape(-1)
    g = s["grad"].float() * s["clip"]
    s["momentum"].mul_(MU).add_(g)
    u = g + MU * s["momentum"] if nesterov else s["momentum"]
    spans = _spans(_shapes(case))[0]
    step = torch.empty_like(u)
    for rows, cols in sorted({(rows, cols) for _, rows, cols in spans}):        # one batch per shape
        alike = [at for at, r, c in spans if (r, c) == (rows, cols)]
        o = _plain_orth(torch.stack([u[at:at + rows * cols].view(rows, cols) for at in alike])).float()
        for at, x in zip(alike, o):
            step[at:at + rows * cols] = x.reshape(-1) * (LR * _scale(rows, cols))
    s["master"].mul_(1 - LR * WD).sub_(step)
    s["param"].copy_(s["master"])
    return {k: s[k] for k in ("master", "momentum", "param")}


# ----------------------------------------------------------------- in 64 bits

def _exact_orth(x):
    """float64 [rows, cols]: each step is an odd polynomial of the singular values, p(X X^T) X, here by Horner's rule on
    the side that has fewer rows."""
    if x.shape[0] > x.shape[1]:
        return _exact_orth(x.t().contiguous()).t()
    x = x / (torch.linalg.vector_norm(x) + EPS)
    for a, b, c in STEPS:
        gram = torch.mm(x, x.t())
        poly = c * gram
        poly.diagonal().add_(b)
        poly = torch.mm(poly, gram)
        poly.diagonal().add_(a)
        x = torch.mm(poly, x)
    return x


def exact(case, seed):
    s = prepare(case, seed)
    spans, total = _spans(_shapes(case))
    if case["op"] == "orth":
        x = s["x"].double()
        return torch.cat([_exact_orth(x[at:at + r * c].view(r, c)).reshape(-1) for at, r, c in spans])
    g = s["grad"].double() * 0.8125
    momentum = MU * s["momentum"].double() + g
    u = g + MU * momentum if case.get("nesterov", True) else momentum
    master = s["master"].double() * (1 - LR * WD)
    for at, r, c in spans:
        master[at:at + r * c] -= LR * _scale(r, c) * _exact_orth(u[at:at + r * c].view(r, c)).reshape(-1)
    return {"master": master, "momentum": momentum, "param": master}
