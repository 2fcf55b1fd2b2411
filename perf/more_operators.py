"""What the orthogonalising optimizer and the relative position bias are measured on.

Four operators, each from one small call to the largest tensors of the repository's models:

  orthogonalize  X = x / (|x| + eps), then five times A = X X^T, X = a X + (b A + c A A) X, for each matrix
  muon           m = mu m + g k, u = g k + mu m, O = orthogonalize(u), w = w (1 - lr wd) - lr scale O, p = bf16(w)
  bias           out[n, h, i, j] = (add[n, h, i, j] or 0) + scale * table[bucket(j - i - start[n]), h]
  bias grad      G[b, h] = (G[b, h] or 0) + scale * sum over n, i, j with bucket(j - i - start[n]) = b of dy[n, h, i, j]

|x| is the Frobenius norm and (a, b, c) = (3.4445, -4.775, 2.0315); matrices with more rows than columns go transposed
(the same values).  bucket(d) with B buckets and the largest distance D: both directions have nb = B / 2 buckets of their
own (those of d > 0 after the others) and take |d|, or one direction has nb = B and takes max(-d, 0); with e = nb / 2 a
distance below e is its own bucket, one from e on is in e + floor(log(distance / e) / log(D / e) * (nb - e)), nb - 1 at most.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}

NS = (3.4445, -4.775, 2.0315)
STEPS, EPS = 5, 1e-7
LR, MU, DECAY = 2e-4, 0.95, 0.1


def _orth(name, count, rows, cols, dtype="bf16"):
    return {"name": name, "op": "orthogonalize", "count": count, "rows": rows, "cols": cols, "dtype": dtype}


def _muon(name, count, rows, cols, lead=0, nesterov=True):
    return {"name": name, "op": "muon", "count": count, "rows": rows, "cols": cols, "lead": lead, "nesterov": nesterov}


def _bias(name, batch, heads, q, k, buckets=32, far=128, both=True, start="0", table="bf16", dtype="bf16", add=True, shift=0):
    return {"name": name, "op": "bias", "batch": batch, "heads": heads, "q": q, "k": k, "buckets": buckets, "far": far, "both": both, "start": start, "table": table, "dtype": dtype, "add": add, "shift": shift}


def _grad(name, batch, heads, q, k, buckets=32, far=128, both=True, start="0", dtype="bf16", grad="f32", accumulate=True, shift=0):
    return {"name": name, "op": "bias grad", "batch": batch, "heads": heads, "q": q, "k": k, "buckets": buckets, "far": far, "both": both, "start": start, "dtype": dtype, "grad": grad, "accumulate": accumulate, "shift": shift}


def listed():
    return [
        # one small matrix: the latency of a call
        _orth("orthogonalize small", 1, 128, 128),
        # GPT-2 small's query, key and value weights of all 12 blocks in one call
        _orth("orthogonalize gpt2 qkv", 12, 768, 2304),
        # odd sizes, more rows than columns, fp32 updates
        _orth("orthogonalize odd", 5, 1531, 777, dtype="f32"),
        # the gate and up weights of a 7B block
        _orth("orthogonalize 7B mlp", 2, 11008, 4096),
        # two blocks' small square weights behind a tensor of odd size: latency, rows at odd places
        _muon("muon small", 4, 96, 160, lead=37, nesterov=False),
        # the attention output weights of the 1.3B model's 24 blocks
        _muon("muon 1.3B proj", 24, 2048, 2048),
        # one gate weight of the 70B shape
        _muon("muon largest", 1, 28672, 8192),
        # one new token of each of 16 sequences of different lengths, added to the scores over a cache: latency
        _bias("bias one token", 16, 12, 1, 1031, both=False, start="each"),
        # a training micro-batch's scores of 2048 positions
        _bias("bias largest", 4, 32, 2048, 2048),
        # odd lengths and heads, fp32, no scores to add to, a table at an odd place of its bucket
        _bias("bias odd", 1, 7, 1531, 3001, buckets=54, far=333, table="f32", dtype="f32", add=False, shift=3),
        # a later micro-batch of GPT-2 small's heads over 1024 positions, causal, into an fp32 bucket
        _grad("bias grad gpt2", 8, 12, 1024, 1024, both=False),
        # 4096 positions in both directions, written to a bf16 bucket
        _grad("bias grad largest", 2, 32, 4096, 4096, far=800, grad="bf16", accumulate=False, shift=5),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v))


def _near_multiple(rng, v):
    m = rng.choice([1, 1, 8, 64, 64, 128])
    return max(1, v // m * m) if v >= m else v


def draw(rng):
    while True:
        op = rng.choice(["orthogonalize", "muon", "bias", "bias grad"])
        if op in ("orthogonalize", "muon"):
            rows, cols = (_near_multiple(rng, _log(rng, 16, 12000)) for _ in range(2))
            count = _log(rng, 1, 48)
            small, large = min(rows, cols), max(rows, cols)
            if count * rows * cols > 100e6 or count * small * small * (2 * large + small) > 2e12:
                continue
            if op == "orthogonalize":
                c = _orth("", count, rows, cols, rng.choice(["bf16", "f32"]))
            else:
                c = _muon("", count, rows, cols, rng.choice([0, 0, 768, rng.randrange(1, 5000)]), rng.random() < 0.7)
        else:
            batch, heads, k = _log(rng, 1, 32), rng.choice([1, 4, 8, 12, 16, 25, 32, 64]), _near_multiple(rng, _log(rng, 8, 8192))
            q = rng.choice([1, k, k, _near_multiple(rng, _log(rng, 2, 4096))])
            if batch * heads * q * k > 5e8:
                continue
            both = rng.random() < 0.5
            buckets = 2 * rng.randrange(4, 65)
            far = _log(rng, buckets, 4000)
            start = "each" if q < k and rng.random() < 0.7 else rng.choice(["0", "end"])
            f = lambda: rng.choice(["bf16", "bf16", "f32"])
            shift = rng.choice([0, 0, 8, rng.randrange(1, 64)])
            if op == "bias":
                c = _bias("", batch, heads, q, k, buckets, far, both, start, f(), f(), rng.random() < 0.7, shift)
            else:
                c = _grad("", batch, heads, q, k, buckets, far, both, start, f(), f(), rng.random() < 0.5, shift)
        del c["name"]
        return c


def _matrices(count, rows, cols, std, gen):
    """Updates as training makes them: a few directions that all samples agree on, over noise of every direction."""
    x = torch.empty(count, rows, cols, device="cuda").normal_(0.0, std, generator=gen)
    r = min(8, rows, cols)
    left = torch.empty(count, rows, r, device="cuda").normal_(0.0, 1.0, generator=gen)
    right = torch.empty(count, r, cols, device="cuda").normal_(0.0, 1.0, generator=gen)
    strength = std * 2.0 ** -torch.arange(r, device="cuda", dtype=torch.float32)
    return x.baddbmm_(left * strength, right)


def _in_buffer(n, dtype, shift, gen, std):
    """n values at place `shift` of a longer flat buffer, as a tensor lies in a bucket."""
    t = torch.empty(n + shift, dtype=TYPES[dtype], device="cuda")
    t.normal_(0.0, std, generator=gen)
    return t[shift:shift + n]


def _start(case, gen):
    """The first query's position among the keys: that of the first key, of the last queries, or each sequence's own."""
    if case["start"] == "0":
        return 0
    if case["start"] == "end":
        return case["k"] - case["q"]
    return torch.randint(0, case["k"] - case["q"] + 1, (case["batch"],), device="cuda", generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] in ("orthogonalize", "muon"):
        count, rows, cols = case["count"], case["rows"], case["cols"]
        n = count * rows * cols
        if case["op"] == "orthogonalize":
            s["x"] = _matrices(count, rows, cols, 1e-3, gen).to(TYPES[case["dtype"]])
            s["out"] = torch.empty(count, rows, cols, dtype=torch.bfloat16, device="cuda")
        else:
            # one bucket of 8 ranks' chunks: `lead` elements of another tensor, then the matrices
            lead, length = case["lead"], -(-(case["lead"] + n) // 512) * 512
            place = slice(lead, lead + n)
            s["master"] = torch.empty(length, device="cuda").normal_(0.0, 0.02, generator=gen)
            s["g"] = torch.zeros(length, device="cuda")
            s["g"][place] = _matrices(count, rows, cols, 1e-3, gen).view(-1)
            s["momentum"] = torch.zeros(length, device="cuda")
            s["momentum"][place] = _matrices(count, rows, cols, 4e-3, gen).view(-1)
            s["params"] = s["master"].bfloat16()
            # the clip coefficient, on the device as the norm's reduction leaves it
            s["coef"] = torch.empty(1, device="cuda").uniform_(0.2, 1.0, generator=gen)
            s["scale"] = 0.2 * math.sqrt(max(rows, cols))
        if own:
            import gradient_sync_zero_amd as G
            s["ws"] = torch.empty(G.muon_workspace_bytes(count, rows, cols), dtype=torch.uint8, device="cuda")
            if case["op"] == "muon":
                s["plan"] = G.Plan([rows * cols] * count + [case["lead"]], 1 << 48, 8)
                s["hp"] = G.make_muon_hp(lr=LR, momentum=MU, weight_decay=DECAY, scale=s["scale"], nesterov=case["nesterov"])
        return s
    batch, heads, q, k = case["batch"], case["heads"], case["q"], case["k"]
    s["start"] = _start(case, gen)
    if case["op"] == "bias":
        s["table"] = _in_buffer(case["buckets"] * heads, case["table"], case["shift"], gen, 0.5).view(case["buckets"], heads)
        s["out"] = torch.empty(batch, heads, q, k, dtype=TYPES[case["dtype"]], device="cuda")
        s["add"] = None
        if case["add"]:
            s["add"] = torch.empty_like(s["out"]).normal_(0.0, 1.0, generator=gen)
            if not case["both"]:  # the future is masked
                s["add"].masked_fill_(_distance(s, case) > 0, -math.inf)
        return s
    s["dy"] = torch.empty(batch, heads, q, k, dtype=TYPES[case["dtype"]], device="cuda").normal_(0.0, 1e-3, generator=gen)
    if not case["both"]:
        s["dy"].masked_fill_(_distance(s, case) > 0, 0.0)
    s["grad"] = _in_buffer(case["buckets"] * heads, case["grad"], case["shift"], gen, 1e-2).view(case["buckets"], heads)
    if own:
        import gradient_sync_zero_amd as G
        s["ws"] = torch.empty(G.relpos_bias_workspace_bytes(batch, heads, q, k, case["buckets"]), dtype=torch.uint8, device="cuda")
    return s


def _distance(s, case):
    """j - i - start[n], as (batch or 1, 1, q, k)."""
    i = torch.arange(case["q"], device="cuda")[:, None]
    j = torch.arange(case["k"], device="cuda")[None, :]
    start = s["start"].view(-1, 1, 1, 1) if isinstance(s["start"], torch.Tensor) else s["start"]
    return (j - i) - start if isinstance(start, torch.Tensor) else (j - i - start)[None, None]


def _bucket(d, case):
    """The bucket of each distance, in 64 bits; the small term keeps a distance that lies on a border on its own side."""
    nb = case["buckets"] // 2 if case["both"] else case["buckets"]
    e = nb // 2
    dist = d.abs() if case["both"] else (-d).clamp(min=0)
    far = e + torch.floor(torch.log(dist.clamp(min=1).double() / e) / math.log(case["far"] / e) * (nb - e) + 1e-9).long()
    b = torch.where(dist < e, dist, far.clamp(max=nb - 1))
    return b + nb * (d > 0) if case["both"] else b


def _orthogonal(x):
    """Newton-Schulz on (count, rows, cols) in fp32."""
    turned = x.shape[1] > x.shape[2]
    x = x.mT.contiguous() if turned else x
    x = x / (x.double().square().sum((1, 2), keepdim=True).sqrt() + EPS).float()
    a, b, c = NS
    for _ in range(STEPS):
        gram = torch.bmm(x, x.mT.contiguous())
        x = a * x + torch.bmm(b * gram + c * torch.bmm(gram, gram), x)
    return x.mT if turned else x


def _plain(s):
    case = s["case"]
    if case["op"] == "orthogonalize":
        return s["out"].copy_(_orthogonal(s["x"].float()))
    if case["op"] == "muon":
        count, rows, cols = case["count"], case["rows"], case["cols"]
        w, m, g, p = (s[k][case["lead"]:case["lead"] + count * rows * cols].view(count, rows, cols) for k in ("master", "momentum", "g", "params"))
        g = g * s["coef"]
        m.copy_(MU * m + g)
        o = _orthogonal(g + MU * m if case["nesterov"] else m)
        w.copy_(w * (1.0 - LR * DECAY) - (LR * s["scale"]) * o)
        p.copy_(w)
        return s["master"], s["momentum"], s["params"]
    if case["op"] == "bias":
        q, k = case["q"], case["k"]
        bias = s["table"].float()[_bucket(_distance(s, case), case).squeeze(1)].permute(0, 3, 1, 2)
        return s["out"].copy_(bias if s["add"] is None else s["add"].float() + bias)
    # each diagonal's sum: rows in reverse order, each followed by q zeros and read one element shorter, have a diagonal as a column
    batch, heads, q, k = s["dy"].shape
    rows = torch.cat([s["dy"].flip(2), s["dy"].new_zeros(batch, heads, q, q)], 3).view(batch, heads, -1)
    sums = rows[:, :, :q * (k + q - 1)].view(batch, heads, q, k + q - 1).sum(2, dtype=torch.float64)
    d = torch.arange(k + q - 1, device="cuda")[None] - (q - 1)
    d = d - (s["start"][:, None] if isinstance(s["start"], torch.Tensor) else s["start"])
    which = (_bucket(d, case)[:, :, None] == torch.arange(case["buckets"], device="cuda")).double().expand(batch, -1, -1).contiguous()
    total = torch.bmm(sums, which).sum(0).T
    return s["grad"].copy_(s["grad"].double() + total if case["accumulate"] else total)


def run(state):
    if not own:
        return _plain(state)
    import gradient_sync_zero_amd as G
    s, case = state, state["case"]
    if case["op"] == "orthogonalize":
        G.orthogonalize(s["x"], s["out"], s["ws"], steps=STEPS, eps=EPS)
        return s["out"]
    if case["op"] == "muon":
        G.muon_step(s["plan"], range(case["count"]), case["rows"], case["cols"], s["master"], s["momentum"], s["g"], s["coef"], s["hp"], s["params"], s["ws"])
        return s["master"], s["momentum"], s["params"]
    if case["op"] == "bias":
        G.relpos_bias(s["table"], s["out"], case["far"], bidirectional=case["both"], q_start=s["start"], add=s["add"])
        return s["out"]
    G.relpos_bias_grad(s["dy"], s["grad"], s["ws"], case["far"], bidirectional=case["both"], q_start=s["start"], accumulate=case["accumulate"])
    return s["grad"]


def work(case):
    if case["op"] in ("orthogonalize", "muon"):
        # the products A and A A are symmetric: half of each; a fused multiply-add counts two
        n = float(case["count"] * case["rows"] * case["cols"])
        small, large = float(min(case["rows"], case["cols"])), float(max(case["rows"], case["cols"]))
        flops = STEPS * case["count"] * (small * small * large + small ** 3 + 2 * small * small * large)
        return {"bytes": n * (SIZE[case["dtype"]] + 2 if case["op"] == "orthogonalize" else 22), "flops": flops}
    n = float(case["batch"] * case["heads"] * case["q"] * case["k"])
    cells = float(case["buckets"] * case["heads"])
    if case["op"] == "bias":
        return {"bytes": n * SIZE[case["dtype"]] * (1 + case["add"]) + cells * SIZE[case["table"]], "flops": n}
    return {"bytes": n * SIZE[case["dtype"]] + cells * SIZE[case["grad"]] * (1 + case["accumulate"]), "flops": n}


def _exact_orthogonal(x):
    """One matrix at a time, each step by Horner's rule from the side of the smaller Gram matrix."""
    out = torch.empty_like(x)
    for k in range(x.shape[0]):
        y = x[k] / (torch.linalg.vector_norm(x[k]) + 1e-7)
        for _ in range(5):
            if y.shape[0] <= y.shape[1]:
                gram = torch.mm(y, y.T)
                y = 3.4445 * y + torch.mm(gram, torch.addmm(y, gram, y, beta=-4.775, alpha=2.0315))
            else:
                gram = torch.mm(y.T, y)
                y = 3.4445 * y + torch.mm(torch.addmm(y, y, gram, beta=-4.775, alpha=2.0315), gram)
        out[k] = y
    return out


def _exact_bucket(d, case):
    """The borders as whole numbers: distance n is past border k of L where n^L e^k >= D^k e^L."""
    half = case["buckets"] // 2 if case["both"] else case["buckets"]
    e = half // 2
    steps = half - e
    borders, n = list(range(1, e + 1)), e
    for k in range(1, steps):
        while n ** steps * e ** k < case["far"] ** k * e ** steps:
            n += 1
        borders.append(n)
    borders = torch.tensor(borders, device="cuda")
    past = torch.searchsorted(borders, d.abs() if case["both"] else -d, right=True)
    return torch.where(d > 0, past + half, past) if case["both"] else past


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "orthogonalize":
        return _exact_orthogonal(s["x"].double())
    if case["op"] == "muon":
        count, rows, cols = case["count"], case["rows"], case["cols"]
        inside = slice(case["lead"], case["lead"] + count * rows * cols)
        w, m = s["master"].double(), s["momentum"].double()
        g = s["g"][inside].double() * s["coef"].double()
        m[inside] = m[inside] * MU + g
        o = _exact_orthogonal((g + m[inside] * MU if case["nesterov"] else m[inside]).view(count, rows, cols)).view(-1)
        w[inside] -= LR * (DECAY * w[inside] + s["scale"] * o)
        p = w.clone()
        outside = torch.ones_like(p, dtype=torch.bool)
        outside[inside] = False
        p[outside] = s["params"][outside].double()
        return w, m, p
    if case["op"] == "bias":
        per_head = s["table"].double().T
        out = s["out"].double()
        for n in range(case["batch"]):
            start = int(s["start"][n]) if isinstance(s["start"], torch.Tensor) else s["start"]
            line = torch.arange(case["k"] + case["q"] - 1, device="cuda") - (case["q"] - 1) - start
            values = per_head[:, _exact_bucket(line, case)]
            # row i reads the stretch of diagonals that begins q - 1 - i places on
            out[n] = values.unfold(1, case["k"], 1).flip(1)
        return out if s["add"] is None else out.add_(s["add"])
    total = s["grad"].double() if case["accumulate"] else torch.zeros_like(s["grad"], dtype=torch.float64)
    for n in range(case["batch"]):
        start = int(s["start"][n]) if isinstance(s["start"], torch.Tensor) else s["start"]
        i, j = torch.arange(case["q"], device="cuda")[:, None], torch.arange(case["k"], device="cuda")[None]
        which = _exact_bucket(j - i - start, case).view(-1)
        order = torch.argsort(which)
        lengths = torch.bincount(which, minlength=case["buckets"])
        for h in range(case["heads"]):
            values = s["dy"][n, h].double().view(-1)[order]
            total[:, h] += torch.segment_reduce(values, "sum", lengths=lengths, unsafe=True, initial=0.0)
    return total
