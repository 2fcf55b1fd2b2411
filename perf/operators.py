"""What the embedding operators and the counter-based dropout are measured on.

Three operators, each from one token to the largest batch a rank of the repository's models holds:

  lookup   out[i, c] = c0 * table[ids[i], c], dropped where the generator says so, 0 where ids[i] is no row
  grad     G[v, c] = (G[v, c] or 0) + c0 * sum over i with ids[i] = v of the kept dy[i, c]
  dropout  y[e] = (add[e] or 0) + (0 if dropped else x[e] * k)

The generator is Philox4x32-10 with key = the two words of the seed and counter = (low and high word of
e >> 3, site, step); element e takes the 16-bit half e & 7 of the four words as the high half of a 32-bit
number and the same half at the counter with the top bit of word 1 set as its low half, and is dropped where
that number is below T = floor(p 2^32).  k = 1 / (1 - T 2^-32), c0 = scale * k, each formed in double.
e is the flat position i * dim + c.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "i32": torch.int32, "i64": torch.int64}
SIZE = {"bf16": 2, "f32": 4, "i32": 4, "i64": 8}

SITE = 7


def _lookup(name, n, dim, rows, ids="zipf", table="bf16", out="bf16", id_type="i64", scale=1.0, p=0.0, shift=0):
    return {"name": name, "op": "lookup", "n": n, "dim": dim, "rows": rows, "ids": ids, "table": table, "out": out, "id_type": id_type, "scale": scale, "p": p, "shift": shift}


def _grad(name, n, dim, rows, ids="zipf", dy="bf16", grad="bf16", id_type="i64", accumulate=False, scale=1.0, p=0.0, shift=0):
    return {"name": name, "op": "grad", "n": n, "dim": dim, "rows": rows, "ids": ids, "dy": dy, "grad": grad, "id_type": id_type, "accumulate": accumulate, "scale": scale, "p": p, "shift": shift}


def _dropout(name, n, dtype="bf16", add=False, p=0.1, shift=0):
    return {"name": name, "op": "dropout", "n": n, "dtype": dtype, "add": add, "p": p, "shift": shift}


def listed():
    return [
        # one token of a serving step on the 70B shape's table: latency
        _lookup("lookup one token", 1, 8192, 32000),
        # a GPT-2 small micro-batch of 8 sequences of 1024 with its embedding dropout
        _lookup("lookup gpt2 dropout", 8192, 768, 50257, p=0.1),
        # 64 Ki tokens on the 70B shape's table, embeddings scaled by sqrt(dim)
        _lookup("lookup largest", 65536, 8192, 32000, scale=math.sqrt(8192.0)),
        # ragged: padded sequences, an odd width, an fp32 table that starts at an odd place of its flat buffer
        _lookup("lookup odd", 4099, 1531, 10007, ids="padded", table="f32", id_type="i32", scale=0.5, p=0.25, shift=3),
        # a few tokens added into the 70B shape's fp32 bucket: latency
        _grad("grad few tokens", 64, 8192, 32000, grad="f32", id_type="i32", accumulate=True),
        # GPT-2 small's micro-batch, its gradient written whole into a bf16 bucket, the dropout mask drawn again
        _grad("grad gpt2 dropout", 8192, 768, 50257, p=0.1),
        # a later micro-batch of a 1.3B accumulation window in fp32 buckets
        _grad("grad 1.3B accumulate", 16384, 2048, 50304, grad="f32", accumulate=True),
        # 64 Ki tokens on the 70B shape, written whole
        _grad("grad largest", 65536, 8192, 32000, scale=math.sqrt(8192.0)),
        # nine tokens in ten are the same one (an unmasked filler), fp32 in and out, an odd width
        _grad("grad one hot row", 16384, 4097, 32000, ids="hot", dy="f32", grad="f32", shift=1),
        # the residual dropout of 8 tokens of GPT-2 small: latency
        _dropout("dropout small", 8 * 768),
        # the residual dropout of 64 Ki tokens of the 70B shape, added to the residual stream
        _dropout("dropout largest", 65536 * 8192, add=True),
        # fp32 activations of an odd count, half of them dropped, from an odd place of their buffer
        _dropout("dropout odd", 50331653, dtype="f32", p=0.5, shift=1),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["lookup", "grad", "dropout"])
        p = rng.choice([0.0, 0.1, 0.1, round(rng.uniform(0.01, 0.9), 3)])
        shift = rng.choice([0, 0, 0, 8, rng.randrange(1, 64)])
        f = lambda: rng.choice(["bf16", "bf16", "f32"])
        if op == "dropout":
            c = _dropout("", _log(rng, 512, 1 << 29), f(), rng.random() < 0.5, p or 0.1, shift)
        else:
            dim = _log(rng, 64, 8192)
            if rng.random() < 0.7:
                m = rng.choice([64, 128, 256])
                dim = max(m, dim // m * m)
            n, rows = _log(rng, 1, 65536), _log(rng, 256, 262144)
            ids = rng.choice(["zipf", "zipf", "uniform", "padded", "hot"])
            it = rng.choice(["i32", "i64"])
            scale = rng.choice([1.0, math.sqrt(dim), round(rng.uniform(0.1, 4.0), 3)])
            if rows * dim > 32000 * 8192:
                continue
            if op == "lookup":
                c = _lookup("", n, dim, rows, ids, f(), f(), it, scale, p, shift)
            else:
                c = _grad("", n, dim, rows, ids, f(), f(), it, rng.random() < 0.5, scale, p, shift)
        del c["name"]
        if work(c)["bytes"] <= most:
            return c


def _frequencies(case, device):
    """How often each row is drawn: token counts of text fall off like 1 / (rank + 2.7), common tokens
    spread over the table; or every row alike."""
    rows = case["rows"]
    if case["ids"] == "uniform":
        return torch.full((rows,), 1.0 / rows, dtype=torch.float64, device=device)
    rank = (torch.arange(rows, dtype=torch.float64, device=device) * 7919) % rows if rows % 7919 else torch.arange(rows, dtype=torch.float64, device=device)
    f = 1.0 / (rank + 2.7)
    return f / f.sum()


def _make_ids(case, gen):
    n = case["n"]
    cdf = torch.cumsum(_frequencies(case, "cuda"), 0)
    u = torch.rand(n, dtype=torch.float64, device="cuda", generator=gen)
    ids = torch.searchsorted(cdf, u).clamp_(max=case["rows"] - 1)
    if case["ids"] == "hot":
        ids = torch.where(torch.rand(n, device="cuda", generator=gen) < 0.9, torch.full_like(ids, case["rows"] // 3), ids)
    if case["ids"] == "padded":  # sequences of 512, the last third of each without a token
        ids = torch.where(torch.arange(n, device="cuda") % 512 < 341, ids, torch.full_like(ids, -1))
    return ids.to(TYPES[case["id_type"]])


def _in_buffer(n, dtype, shift, gen, std):
    """n values at place `shift` of a longer flat buffer, as a tensor lies in a bucket."""
    t = torch.empty(n + shift, dtype=TYPES[dtype], device="cuda")
    t.normal_(0.0, std, generator=gen)
    return t[shift:shift + n]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    # the generator's seed and the training step, on the device as a step's other scalars are
    s["rng"] = torch.tensor([(seed * 0x9E3779B97F4A7C15 + 12345) & 0x7FFFFFFFFFFFFFFF, seed % 1000], dtype=torch.int64, device="cuda")
    n, shift = case["n"], case["shift"]
    if case["op"] == "dropout":
        s["x"] = _in_buffer(n, case["dtype"], shift, gen, 1.0)
        s["add"] = _in_buffer(n, case["dtype"], 0, gen, 1.0) if case["add"] else None
        s["y"] = torch.empty(n, dtype=TYPES[case["dtype"]], device="cuda")
        return s
    rows, dim = case["rows"], case["dim"]
    s["ids"] = _make_ids(case, gen)
    if case["op"] == "lookup":
        s["table"] = _in_buffer(rows * dim, case["table"], shift, gen, 0.02).view(rows, dim)
        s["out"] = torch.empty(n, dim, dtype=TYPES[case["out"]], device="cuda")
    else:
        s["dy"] = _in_buffer(n * dim, case["dy"], 0, gen, 1e-3).view(n, dim)
        s["grad"] = _in_buffer(rows * dim, case["grad"], shift, gen, 1e-3).view(rows, dim)
        if own:
            import gradient_sync_zero_amd as G
            s["ws"] = torch.empty(G.embedding_workspace_bytes(n, rows, dim) // 8, dtype=torch.float64, device="cuda")
    return s


def _threshold(p):
    return math.floor(p * 2.0 ** 32)


def _keep_scale(p):
    return 1.0 / (1.0 - _threshold(p) * 2.0 ** -32)


def _philox(c0, c1, c2, c3, k0, k1):
    """Ten rounds on int64 tensors that hold 32-bit words; a product of two words wraps mod 2^64, and the mask takes its high word."""
    m = 0xFFFFFFFF
    for r in range(10):
        a, b = 0xD2511F53 * c0, 0xCD9E8D57 * c2
        key0, key1 = (k0 + r * 0x9E3779B9) & m, (k1 + r * 0xBB67AE85) & m
        c0, c1, c2, c3 = ((b >> 32) & m) ^ c1 ^ key0, b & m, ((a >> 32) & m) ^ c3 ^ key1, a & m
    return torch.stack([c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16, c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16], 1).reshape(-1)


def _kept(n, p, rng):
    """Which of the elements [0, n) are kept."""
    m = 0xFFFFFFFF
    block = torch.arange((n + 7) // 8, dtype=torch.int64, device=rng.device)
    low, high = block & m, block >> 32
    site, step = torch.full_like(block, SITE), (rng[1] & m).expand_as(block)
    k0, k1 = rng[0] & m, (rng[0] >> 32) & m
    u = (_philox(low, high, site, step, k0, k1) << 16) | _philox(low, high | 0x80000000, site, step, k0, k1)
    return u[:n] >= _threshold(p)


def _plain(s):
    case = s["case"]
    p = case["p"]
    if case["op"] == "dropout":
        y = torch.where(_kept(case["n"], p, s["rng"]), s["x"].float() * _keep_scale(p), 0.0)
        return (y if s["add"] is None else s["add"].float() + y).to(s["y"].dtype)
    n, dim, rows = case["n"], case["dim"], case["rows"]
    c0 = case["scale"] * _keep_scale(p)
    ids = s["ids"].long()
    is_row = (ids >= 0) & (ids < rows)
    kept = _kept(n * dim, p, s["rng"]).view(n, dim) & is_row[:, None] if p else is_row[:, None]
    if case["op"] == "lookup":
        return torch.where(kept, s["table"][ids.clamp(0, rows - 1)].float() * c0, 0.0).to(s["out"].dtype)
    total = torch.zeros(rows, dim, dtype=torch.float32, device=ids.device)
    total.index_add_(0, ids.clamp(0, rows - 1), torch.where(kept, s["dy"].float(), 0.0))
    total *= c0
    s["grad"].copy_(s["grad"].float() + total if case["accumulate"] else total)
    return s["grad"]


def run(state):
    if not own:
        return _plain(state)
    import gradient_sync_zero_amd as G
    case = state["case"]
    if case["op"] == "dropout":
        G.dropout(state["x"], state["y"], case["p"], state["rng"], SITE, add=state["add"])
        return state["y"]
    rng = state["rng"] if case["p"] else None
    if case["op"] == "lookup":
        G.embedding_lookup(state["ids"], state["table"], state["out"], scale=case["scale"], p=case["p"], rng=rng, site=SITE)
        return state["out"]
    G.embedding_grad(state["ids"], state["dy"], state["grad"], state["ws"], scale=case["scale"], p=case["p"], rng=rng, site=SITE, accumulate=case["accumulate"])
    return state["grad"]


def _distinct(case):
    """The expected number of distinct rows among the tokens."""
    n, rows = case["n"], case["rows"]
    f = _frequencies(case, "cpu")
    if case["ids"] == "hot":
        n = n * 0.1
    if case["ids"] == "padded":
        n = n * 341 / 512
    seen = float((1.0 - torch.exp(n * torch.log1p(-f.clamp(max=0.999999)))).sum())
    return max(1.0, min(seen + (case["ids"] == "hot"), rows, case["n"]))


def work(case):
    # A Philox block of ten rounds serves eight elements: 20 products of 32 x 32 bits, 40 xors and its
    # selection, counted as 10 operations an element; a scale or an addition counts one.
    n = case["n"]
    drop = 10.0 if case["p"] else 0.0
    if case["op"] == "dropout":
        return {"bytes": float(n * SIZE[case["dtype"]] * (3 if case["add"] else 2)), "flops": n * (drop + 1 + case["add"])}
    dim, rows = case["dim"], case["rows"]
    size = n * SIZE[case["id_type"]]
    if case["op"] == "lookup":
        size += _distinct(case) * dim * SIZE[case["table"]] + n * dim * SIZE[case["out"]]
        return {"bytes": float(size), "flops": float(n * dim * (drop + 1))}
    size += n * dim * SIZE[case["dy"]]
    size += (2 * _distinct(case) if case["accumulate"] else rows) * dim * SIZE[case["grad"]]
    return {"bytes": float(size), "flops": float(n * dim * (drop + 1))}


def _exact_kept(n, p, rng):
    """The generator once more, its high words put together from 16-bit parts."""
    seed, step = int(rng[0]), int(rng[1])

    def product(m, x):
        ml, mh, xl, xh = m & 0xFFFF, m >> 16, x & 0xFFFF, x >> 16
        low = ml * xl
        mid = ml * xh + (low >> 16)
        mid2 = mh * xl + (mid & 0xFFFF)
        return mh * xh + (mid >> 16) + (mid2 >> 16), ((mid2 & 0xFFFF) << 16) | (low & 0xFFFF)

    def words(top, first, last):
        e = torch.arange(first, last, dtype=torch.int64, device="cuda")
        x = [e % 2 ** 32, e // 2 ** 32 + top, torch.full_like(e, SITE), torch.full_like(e, step % 2 ** 32)]
        key = [seed % 2 ** 32, seed // 2 ** 32 % 2 ** 32]
        for _ in range(10):
            (h0, l0), (h1, l1) = product(0xD2511F53, x[0]), product(0xCD9E8D57, x[2])
            x = [h1 ^ x[1] ^ key[0], l1, h0 ^ x[3] ^ key[1], l0]
            key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
        return torch.stack(x, 1)

    kept = torch.empty((n + 7) // 8 * 8, dtype=torch.bool, device="cuda")
    for first in range(0, (n + 7) // 8, 1 << 22):
        last = min(first + (1 << 22), (n + 7) // 8)
        a, b = words(0, first, last), words(2 ** 31, first, last)
        low = (a % 65536) * 65536 + b % 65536
        high = (a // 65536) * 65536 + b // 65536
        kept[8 * first:8 * last] = ~(torch.stack([low, high], 2).reshape(-1).double() < math.floor(p * 2.0 ** 32))
    return kept[:n]


def exact(case, seed):
    s = prepare(case, seed)
    p, n = case["p"], case["n"]
    k = 1.0 / (1.0 - math.floor(p * 2.0 ** 32) / 2.0 ** 32)
    if case["op"] == "dropout":
        y = s["x"].double() * k
        y[~_exact_kept(n, p, s["rng"])] = 0.0
        return y if s["add"] is None else y.add_(s["add"])
    rows, dim, ids = case["rows"], case["dim"], s["ids"].long()
    gone = ~_exact_kept(n * dim, p, s["rng"]).view(n, dim) if p else None
    none = (ids < 0) | (ids >= rows)
    if case["op"] == "lookup":
        out = s["table"].double().index_select(0, ids.masked_fill(none, 0)) * (case["scale"] * k)
        out[none] = 0.0
        return out if gone is None else out.masked_fill_(gone, 0.0)
    # rows of one token are neighbours after a sort; the sum of each run is taken in slices of columns
    order = torch.argsort(ids.masked_fill(none, rows), stable=True)
    order = order[:n - int(none.sum())]
    run = ids[order]
    total = torch.empty(rows, dim, dtype=torch.float64, device="cuda")
    for c in range(0, dim, 512):
        part = s["dy"][:, c:c + 512].double()
        if gone is not None:
            part.masked_fill_(gone[:, c:c + 512], 0.0)
        sums = torch.segment_reduce(part[order], "sum", lengths=torch.bincount(run, minlength=rows), axis=0, unsafe=True, initial=0.0)
        total[:, c:c + 512] = sums * (case["scale"] * k)
    return total.add_(s["grad"]) if case["accumulate"] else total
