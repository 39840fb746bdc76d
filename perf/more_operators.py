"""Workloads of two sets of operators that belong together: the head that makes
rows of logits, and the draws that are made from rows.

A model's head is a matrix product whose weights are kept in 8 bits with a scale
for each block of 128; it makes the rows of real logits that the framework's
operators on outcome distributions score and train on.  Outcomes are then drawn
from such rows, or from rows of amplitudes, which is what a contraction with open
modes is run for.  This file runs each operator in its plain form (elementary
torch operations) and through the framework's calls (``own``):

``sample``       outcomes drawn from rows by given random numbers, with
                 temperature, top-k, top-p and min-p
``quantize``     a matrix in 8 bits: codes and a scale for each block of 128
``linear``       y = Q(x) Q(W)^T from the 8-bit weights
``linear_grad``  its gradients dx = Q(dy) Q(W) and dW = Q'(dy)^T Q'(x), where Q'
                 has its blocks along the rows that are summed over

Definitions of the draws.  The logit of an entry is the real entry, or ln w with w =
re^2 + im^2 (each operation rounded to 32 bits) for an amplitude; an entry is
absent where the mask is zero or its logit is -inf.  With c = scale / temperature
(one division in 32 bits) an entry's weight is exp(c z).  Three filters follow each
other: the top_k entries of largest logit (ties to the lowest index, 0: all), of
those the shortest run of largest ones whose weight is top_p of theirs at least (1:
all), of those the ones whose weight is min_p of the largest at least (0: all).  A
draw with the number u is the first entry left, in the order of indices, up to which the
weights' sum exceeds u times that of all left.  logp is the logarithm of its
probability among those, and kept is how many there are.  A temperature of 0 leaves the
largest entry.  The parameters are numbers of 32 bits.  A row without entries has outcome -1, log p -inf and kept 0.  The plain
form is in 64 bits, as sums next to a border decide here.

Definitions of the codes.  A block is 128 entries of a row (the last may be
shorter), or 128 x 128 entries for weights.  Its scale s is the smallest power of
two from 2^-126 on for which max |x| / s <= 448 (1 for a block of zeros), its codes
are x / s rounded to e4m3 (ties to even).
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"c64": torch.complex64, "f32": torch.float32, "bf16": torch.bfloat16,
          "f16": torch.float16}
_BYTES = {"c64": 8, "f32": 4, "bf16": 2, "f16": 2}
_F8 = torch.float8_e4m3fn


def _sample(name, type_, rows, cols, draws=1, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0,
            each=False, mask=False, scale=1.0, wide=False):
    """each: parameters of every row's own, around the given ones; wide: u in 64 bits."""
    return {"name": name, "op": "sample", "type": type_, "rows": rows, "cols": cols, "draws": draws,
            "temperature": temperature, "top_k": top_k, "top_p": top_p, "min_p": min_p, "each": each,
            "mask": mask, "scale": scale, "wide": wide}


def _quantize(name, type_, rows, cols, square=False, layout="rows"):
    """square: blocks of 128 x 128; layout: rows, columns (the transposed matrix) or both."""
    return {"name": name, "op": "quantize", "type": type_, "rows": rows, "cols": cols,
            "square": square, "layout": layout}


def _linear(name, op, type_, rows, outs, cols, result):
    """rows tokens, outs outcomes, cols features; result: type of y or of dW."""
    return {"name": name, "op": op, "type": type_, "rows": rows, "outs": outs, "cols": cols,
            "result": result}


def listed():
    return [
        # one new token of one sequence, with the usual filters; all latency
        _sample("sample_one_token", "bf16", 1, 32768, temperature=0.75, top_k=40, top_p=0.9375),
        # a decoding batch over a large vocabulary, every request with its own nucleus
        _sample("sample_decode_batch", "bf16", 64, 131072, temperature=0.875, top_p=0.9, min_p=0.002,
                each=True),
        # rollouts for training, without filters, over an odd vocabulary; grammar masks
        _sample("sample_rollout_odd", "f16", 1024, 50001, temperature=1.25, mask=True),
        # thousands of shots of the state of 24 open qubits
        _sample("sample_shots", "c64", 1, 1 << 24, draws=4096, wide=True),
        # one shot each of six open qubits for many projections
        _sample("sample_six_qubits", "c64", 20000, 64),
        # activations on their way into a product
        _quantize("quantize_activations", "bf16", 4096, 4096),
        # weights of an odd vocabulary after an optimiser's step, for both directions
        _quantize("quantize_weights", "f32", 50001, 2048, square=True, layout="both"),
        # the head for one token: the weights' bytes
        _linear("linear_one_token", "linear", "bf16", 1, 32768, 4096, "f32"),
        # the head for a decoding batch over an odd vocabulary
        _linear("linear_decode_batch", "linear", "bf16", 48, 50001, 2048, "bf16"),
        # the head for a prompt or a training batch
        _linear("linear_prompt", "linear", "bf16", 4096, 32768, 4096, "bf16"),
        # a training batch's backward pass
        _linear("linear_grad", "linear_grad", "bf16", 4096, 16384, 4096, "f32"),
        # ragged in every side
        _linear("linear_grad_odd", "linear_grad", "f16", 1000, 5003, 1112, "f32"),
    ]


_MOST_FLOPS = 2 * 4096 * 32768 * 4096       # of one product of the largest listed case


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(max(v, lo), hi)


def draw(rng):
    op = rng.choice(["sample", "sample", "sample", "quantize", "linear", "linear", "linear_grad"])
    if op == "sample":
        type_ = rng.choice(["bf16", "bf16", "f16", "f32", "c64"])
        kind = rng.random()
        draws = 1
        if kind < 0.2:          # few outcomes, many rows
            cols, rows = _log_int(rng, 1, 2048), _log_int(rng, 1, 50000)
        elif kind < 0.4:        # a long row or a few, and shots
            cols, rows, draws = _log_int(rng, 1 << 17, 1 << 24), _log_int(rng, 1, 4), _log_int(rng, 1, 4096)
        else:
            cols, rows = _log_int(rng, 2048, 1 << 18), _log_int(rng, 1, 1024)
            draws = rng.choice([1, 1, 1, 2, 16])
        if rng.random() < 0.5:  # aligned rows in one half of the draws
            cols = max(16, cols // 16 * 16)
        rows = max(1, min(rows, (1 << 25) // cols))
        return {"op": op, "type": type_, "rows": rows, "cols": cols, "draws": draws,
                "temperature": rng.choice([1.0, 1.0, 0.75, 0.5, 1.25]),
                "top_k": rng.choice([0, 0, 0, 1, 20, 64, 1000, 5000]),
                "top_p": rng.choice([1.0, 1.0, 0.5, 0.9, 0.95]),
                "min_p": rng.choice([0.0, 0.0, 0.05, 0.001]),
                "each": rng.random() < 0.5, "mask": rng.random() < 0.3,
                "scale": rng.choice([1.0, 1.0, 0.5]), "wide": type_ == "c64" or rng.random() < 0.2}
    type_ = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "quantize":
        rows, cols = _log_int(rng, 1, 32768), _log_int(rng, 1, 16384)
        return {"op": op, "type": type_, "rows": max(1, min(rows, (1 << 26) // cols)), "cols": cols,
                "square": rng.random() < 0.4, "layout": rng.choice(["rows", "columns", "both"])}
    rows, outs, cols = _log_int(rng, 1, 8192), _log_int(rng, 128, 65536), _log_int(rng, 64, 8192)
    if rng.random() < 0.5:
        outs, cols = outs // 128 * 128, max(128, cols // 128 * 128)
    most = _MOST_FLOPS // (2 if op == "linear_grad" else 1) // 2
    rows = max(1, min(rows, most // (outs * cols), (1 << 27) // outs))
    return {"op": op, "type": type_, "rows": rows, "outs": outs, "cols": cols,
            "result": rng.choice(["f32", type_])}


# ---- inputs -----------------------------------------------------------------

def _sample_inputs(case, gen):
    R, V, t = case["rows"], case["cols"], case["type"]

    def rand(*shape, dtype=torch.float32):
        return torch.rand(shape, generator=gen, device="cuda", dtype=dtype)
    f = {}
    if t == "c64":
        # a random circuit's amplitudes with ten more qubits projected
        f["rows"] = torch.view_as_complex(
            torch.randn((R, V, 2), generator=gen, device="cuda") * (0.5 / V / 1024) ** 0.5)
    else:
        # logits of a trained head: a broad normal body, and each row its own sharpness
        z = torch.randn((R, V), generator=gen, device="cuda")
        f["rows"] = (z * (1.0 + 2.0 * rand(R, 1))).to(_TYPES[t])
        del z
    f["mask"] = None
    if case["mask"]:
        mask = rand(R, V) < rand(R, 1)
        if R >= 8:
            mask[R // 2] = False          # a row that the mask leaves empty
        f["mask"] = mask
        bad = rand(R, V) < 0.01           # what lies in masked places is left over
        f["rows"][bad & ~mask] = float("nan")
        del bad
    f["u"] = rand(R, case["draws"], dtype=torch.float64 if case["wide"] else torch.float32)
    for name in ("temperature", "top_k", "top_p", "min_p"):
        f[name] = case[name]
    if case["each"]:
        # every request its own: some greedy, some without this or that filter
        keep = rand(4, R)
        f["temperature"] = torch.where(keep[0] < 0.9, case["temperature"] * (0.75 + 0.5 * rand(R)), 0.0)
        if case["top_k"]:
            k = 1 + (rand(R) * 2 * case["top_k"]).int()
            f["top_k"] = torch.where(keep[1] < 0.8, k, 0)
        if case["top_p"] < 1.0:
            f["top_p"] = torch.where(keep[2] < 0.8, case["top_p"] + (rand(R) - 0.5) * 0.0625, 1.0)
        if case["min_p"]:
            f["min_p"] = torch.where(keep[3] < 0.8, case["min_p"] * 2 * rand(R), 0.0)
    return f


def _matrix(gen, rows, cols, type_, width=1.0):
    """Activations or gradients: normal entries, some features far larger than others,
    a few tokens of zeros (padding)."""
    x = torch.randn((rows, cols), generator=gen, device="cuda") * width
    x *= torch.exp(torch.randn((1, cols), generator=gen, device="cuda") * 0.75)
    x *= (torch.rand((rows, 1), generator=gen, device="cuda") > 0.02).float()
    return x.to(_TYPES[type_])


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 6007 + 29)
    if case["op"] == "sample":
        return _sample_inputs(case, gen)
    if case["op"] == "quantize":
        return {"x": _matrix(gen, case["rows"], case["cols"], case["type"])}
    f = {"x": _matrix(gen, case["rows"], case["cols"], case["type"])}
    if case["op"] == "linear_grad":
        f["dy"] = _matrix(gen, case["rows"], case["outs"], case["type"], 2.0 ** -10)
    f["w"] = torch.randn((case["outs"], case["cols"]), generator=gen, device="cuda") * case["cols"] ** -0.5
    return f


def _padded(codes):
    """The codes with rows that start at multiples of 16 bytes, as the calls take them."""
    pad = torch.zeros((codes.shape[0], (codes.shape[1] + 15) // 16 * 16), dtype=torch.uint8,
                      device=codes.device).view(_F8)
    pad.view(torch.uint8)[:, :codes.shape[1]] = codes.view(torch.uint8)
    return pad[:, :codes.shape[1]]


def prepare(case, seed):
    f = _inputs(case, seed)
    f["case"] = dict(case)
    if case["op"] == "sample" and own:
        import exact_tensor_network_gb300 as tn
        f["op"] = tn.Sampler(case["cols"], _TYPES[case["type"]], max_rows=case["rows"],
                             draws=case["draws"], scale=case["scale"])
        f["op"].bind_workspace()
    if case["op"].startswith("linear"):
        # the weights as a program keeps them: 8 bits, for a backward pass transposed
        w = f.pop("w")
        codes, scales = _plain_codes(w.t() if case["op"] == "linear_grad" else w, True)
        f["codes"], f["scales"] = _padded(codes), scales.contiguous()
    return f


# ---- the plain forms --------------------------------------------------------

_NEG = float("-inf")


def _plain_sample(s):
    c, rows, mask, u = s["case"], s["rows"], s["mask"], s["u"]
    R, V = rows.shape

    def each(v, dtype):
        return torch.as_tensor(v, dtype=dtype, device=rows.device).expand(R)[:, None]
    temperature = each(s["temperature"], torch.float32)
    greedy = temperature == 0
    beta = (c["scale"] / torch.where(greedy, 1.0, temperature)).double()
    if rows.is_complex():
        order = rows.real * rows.real + rows.imag * rows.imag
        z = torch.log(order.double())
    else:
        order = rows.float() + 0.0
        z = order.double()
    present = z != _NEG
    if mask is not None:
        present = present & mask
    x = torch.where(present, z * beta, _NEG)
    m = x.amax(dim=1, keepdim=True)
    m = torch.where(m == _NEG, 0.0, m)
    w = torch.exp(x - m)
    if rows.is_complex():       # amplitudes' own weights need no logarithm
        w = torch.where(beta == 1.0, torch.where(present, order.double(), 0.0), w)
    bad = torch.isnan(m)
    del x, z
    keep = present
    k, p, least = each(s["top_k"], torch.int64), each(s["top_p"], torch.float32).double(), each(s["min_p"], torch.float32).double()
    if s["case"]["top_k"] or s["case"]["top_p"] < 1.0 or s["case"]["each"]:
        bits = order.contiguous().view(torch.int32)
        bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
        key = (bits << 32) | (V - 1 - torch.arange(V, device=bits.device))
        key = torch.where(present, key, torch.iinfo(torch.int64).min)
        del bits
        at = torch.sort(key, dim=1, descending=True).indices
        del key
        rank = torch.arange(V, device=at.device)[None, :]
        ws = torch.where((rank < k) | (k <= 0), w.gather(1, at), 0.0)
        ws = torch.where(greedy & (rank > 0), 0.0, ws)
        before = torch.cumsum(ws, dim=1)
        total = before[:, -1:].clone()
        before -= ws
        stays = (ws > 0) & ((before < p * total) | (p >= 1) | (rank == 0))
        keep = torch.zeros_like(present).scatter_(1, at, stays)
        del at, ws, before, stays
    keep = keep & (w >= least * w.amax(dim=1, keepdim=True))
    w = torch.where(keep, w, 0.0)
    cdf = torch.cumsum(w, dim=1)
    total = cdf[:, -1:]
    aim = u.double() * total
    ids = torch.searchsorted(cdf, aim, right=True).clamp(max=V - 1)
    pick = w.gather(1, ids)
    logp = torch.log(pick / total)
    none = ~keep.any(dim=1, keepdim=True) | bad
    ids = torch.where(none, -1, ids)
    logp = torch.where(bad, float("nan"), torch.where(none, _NEG, logp))
    return {"ids": ids, "logp": logp.float(), "kept": torch.where(none[:, 0], 0, keep.sum(dim=1))}


def _plain_scale(top):
    """The smallest power of two s with top / s <= 448."""
    m, e = torch.frexp(top)                 # top = m 2^e, 0.5 <= m < 1; 448 = 0.875 2^9
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126)
    return torch.where(top == 0, 1.0, torch.ldexp(torch.ones_like(top), e))


def _plain_blocks(x, square):
    """The matrix in 32 bits, padded to whole blocks: [row blocks, rows, blocks, 128]."""
    R, C = x.shape
    r = 128 if square else 1
    x = torch.nn.functional.pad(x.float(), (0, -C % 128, 0, -R % r))
    return x.reshape(x.shape[0] // r, r, x.shape[1] // 128, 128)


def _plain_codes(x, square):
    """Codes [R, C] and scales [R or R / 128, C / 128]."""
    b = _plain_blocks(x, square)
    s = _plain_scale(b.abs().amax(dim=(1, 3)))
    q = (b / s[:, None, :, None]).to(_F8)
    return q.view(torch.uint8).reshape(b.shape[0] * b.shape[1], -1).view(_F8)[:x.shape[0], :x.shape[1]], s


def _plain_values(codes, scales, square):
    b = _plain_blocks(codes, square) * scales[:, None, :, None]
    return b.reshape(b.shape[0] * b.shape[1], -1)[:codes.shape[0], :codes.shape[1]]


def _plain_quantized(x, square):
    """What the codes stand for."""
    return _plain_values(*_plain_codes(x, square), square)


def _plain(s):
    c = s["case"]
    if c["op"] == "sample":
        return _plain_sample(s)
    x, out = s["x"], {}
    if c["op"] == "quantize":
        for layout, m in (("rows", x), ("columns", x.t())):
            if c["layout"] in (layout, "both"):
                codes, scales = _plain_codes(m, c["square"])
                out[layout] = {"codes": codes, "scales": scales}
        return out
    w = _plain_values(s["codes"], s["scales"], True)
    if c["op"] == "linear":
        return {"y": (_plain_quantized(x, False) @ w.t()).to(_TYPES[c["result"]])}
    dy = s["dy"]
    dx = _plain_quantized(dy, False) @ w.t()
    dw = _plain_quantized(dy.t(), False) @ _plain_quantized(x.t(), False).t()
    return {"dx": dx.to(_TYPES[c["type"]]), "dw": dw.to(_TYPES[c["result"]])}


# ---- one pass ---------------------------------------------------------------

def run(s):
    if not own:
        return _plain(s)
    import exact_tensor_network_gb300 as tn
    c = s["case"]
    if c["op"] == "sample":
        r = s["op"].sample(s["rows"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                           top_p=s["top_p"], min_p=s["min_p"], mask=s["mask"])
        return {"ids": r.ids, "logp": r.logp, "kept": r.kept}
    if c["op"] == "quantize":
        got = tn.quantize8(s["x"], square=c["square"], layout=c["layout"])
        if c["layout"] != "both":
            got = (got,)
        names = ("rows", "columns") if c["layout"] == "both" else (c["layout"],)
        return {n: {"codes": b.codes, "scales": b.scales} for n, b in zip(names, got)}
    w = tn.Blocks8(s["codes"], s["scales"])
    if c["op"] == "linear":
        return {"y": tn.linear8(s["x"], w, dtype=_TYPES[c["result"]])}
    dx, dw = tn.linear8_grad(s["x"], s["dy"], w, dtype=_TYPES[c["result"]])
    return {"dx": dx, "dw": dw}


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    if case["op"] == "sample":
        R, V, D = case["rows"], case["cols"], case["draws"]
        n = R * V
        moved = n * _BYTES[case["type"]] + (n if case["mask"] else 0)
        moved += R * D * ((8 if case["wide"] else 4) + 12) + 8 * R + (16 * R if case["each"] else 0)
        return {"bytes": moved, "flops": (8 if case["type"] == "c64" else 5) * n}
    R, C, b = case["rows"], case["cols"], _BYTES[case["type"]]

    def codes(rows, cols, square):
        return rows * cols + 4 * (-(-rows // 128) if square else rows) * -(-cols // 128)
    if case["op"] == "quantize":
        moved = R * C * b
        if case["layout"] != "columns":
            moved += codes(R, C, case["square"])
        if case["layout"] != "rows":
            moved += codes(C, R, case["square"])
        return {"bytes": moved, "flops": 3 * R * C}
    N, out = case["outs"], _BYTES[case["result"]]
    moved = R * C * b + codes(N, C, True)
    if case["op"] == "linear":
        return {"bytes": moved + R * N * out, "flops": 2 * R * N * C}
    return {"bytes": moved + R * N * b + R * C * b + N * C * out, "flops": 4 * R * N * C}


# ---- the definitions in 64 bits ---------------------------------------------

def _exact_sample_block(case, f, lo, hi):
    a = f["rows"][lo:hi]
    n, V = a.shape
    inf = float("inf")

    def par(name, dtype):
        v = f[name]
        return v[lo:hi].to(dtype) if torch.is_tensor(v) else torch.full((n,), v, dtype=dtype, device=a.device)
    temp = par("temperature", torch.float32)
    c = torch.where(temp > 0, torch.tensor(case["scale"], device=a.device) / temp, 1.0).double()[:, None]
    if a.is_complex():
        weight32 = torch.add(a.real.contiguous().square(), a.imag.contiguous().square())
        rank_by = weight32.double()
        gone = rank_by == 0
    else:
        rank_by = a.double()
        gone = rank_by.isneginf()
    if f["mask"] is not None:
        gone = gone | f["mask"][lo:hi].logical_not()
    rank_by = rank_by.masked_fill(gone, -inf)
    largest = rank_by.max(dim=1, keepdim=True).values
    undefined = largest.isnan().squeeze(1)
    empty = gone.all(dim=1)
    safe = torch.where(largest.isneginf(), 1.0, largest)
    if a.is_complex():
        rel = torch.pow((rank_by / safe).masked_fill(gone, 0.0), c)
        rel = torch.where(c == 1.0, rank_by.masked_fill(gone, 0.0), rel)
    else:
        rel = torch.exp(c * (rank_by - safe)).masked_fill(gone, 0.0)
    alive = gone.logical_not()
    k = par("top_k", torch.int64)
    k = torch.where(temp == 0, 1, torch.where(k > 0, k, V))
    p, least = par("top_p", torch.float32).double(), par("min_p", torch.float32).double()
    if bool((k < V).any()) or bool((p < 1).any()):
        order = torch.sort(rank_by, dim=1, descending=True, stable=True).indices
        place = torch.empty_like(order).scatter_(1, order, torch.arange(V, device=a.device).expand(n, V).contiguous())
        alive = alive & (place < k[:, None])
        run_ = (rel * alive).gather(1, order)
        upto = run_.cumsum(dim=1)
        # how many of the largest ones it takes
        need = torch.searchsorted(upto, (p * upto[:, -1])[:, None].contiguous()).squeeze(1) + 1
        need = torch.where(p >= 1, V, need)
        alive = alive & (place < need[:, None])
    alive = alive & (rel >= least[:, None] * rel.max(dim=1, keepdim=True).values)
    rel = rel * alive
    upto = rel.cumsum(dim=1)
    z = upto[:, -1:].contiguous()
    at = torch.searchsorted(upto, (f["u"][lo:hi].double() * z).contiguous(), right=True).clamp(max=V - 1)
    logp = rel.gather(1, at).log() - z.log()
    kept = alive.sum(dim=1)
    dead = empty | undefined
    at[dead] = -1
    logp[empty] = -inf
    logp[undefined] = float("nan")
    kept[dead] = 0
    return {"ids": at, "logp": logp, "kept": kept}


def _exact_codes(x, square):
    """(codes' values, scales) in 64 bits, block by block of columns."""
    x = x.double()
    R, C = x.shape
    tall = 128 if square else 1
    codes = torch.empty_like(x)
    scales = torch.empty((-(-R // tall), -(-C // 128)), dtype=torch.float64, device=x.device)
    for j in range(scales.shape[1]):
        cut = x[:, 128 * j:128 * j + 128]
        top = cut.abs().max(dim=1).values
        if square:
            top = torch.stack([t.max() for t in top.split(128)])
        s = torch.exp2(torch.ceil(torch.log2(top / 448.0)).clamp(min=-126.0))
        s = torch.where(top / s > 448.0, s * 2, torch.where(top / (s / 2) <= 448.0, s / 2, s))
        s = torch.where(top == 0, 1.0, s.clamp(min=2.0 ** -126))
        scales[:, j] = s
        v = cut / s.repeat_interleave(tall)[:R, None]
        # the distance of e4m3's neighbours: 2^-3 of the power of two, 2^-9 at the least
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        codes[:, 128 * j:128 * j + 128] = torch.round(v / step) * step
    return codes, scales


def _exact_matrix(x, square):
    codes, scales = _exact_codes(x, square)
    tall = 128 if square else 1
    return codes * scales.repeat_interleave(tall, 0)[:x.shape[0]].repeat_interleave(128, 1)[:, :x.shape[1]]


def exact(case, seed):
    f = _inputs(case, seed)
    if case["op"] == "sample":
        R, V = case["rows"], case["cols"]
        step = max(1, (1 << 24) // V)
        parts = [_exact_sample_block(case, f, lo, min(R, lo + step)) for lo in range(0, R, step)]
        return {k: torch.cat([p[k] for p in parts]).cpu().numpy() for k in parts[0]}
    x = f["x"]
    if case["op"] == "quantize":
        out = {}
        for layout, m in (("rows", x), ("columns", x.t())):
            if case["layout"] in (layout, "both"):
                codes, scales = _exact_codes(m, case["square"])
                out[layout] = {"codes": codes.float().cpu().numpy(), "scales": scales.cpu().numpy()}
        return out
    if case["rows"] * case["outs"] * case["cols"] > 1 << 41:
        return None
    w = _exact_matrix(f["w"], True)
    if case["op"] == "linear":
        return {"y": torch.mm(_exact_matrix(x, False), w.t()).cpu().numpy()}
    dy = f["dy"]
    dx = torch.mm(_exact_matrix(dy, False), w)
    dw = torch.mm(_exact_matrix(dy.t(), False), _exact_matrix(x.t(), False).t())
    return {"dx": dx.cpu().numpy(), "dw": dw.cpu().numpy()}
