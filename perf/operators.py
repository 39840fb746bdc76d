"""Workloads of the operators on outcome distributions.

A contraction with open modes answers with a batch of rows: amplitudes over
the outcomes of the open qubits, or real logits where the network is a
model's head.  Two operators work on such rows, and this file runs each in
its plain form (elementary torch operations in 32 bits) and through the
framework's calls (``own``):

``score``         log probabilities of given outcomes, the row's log
                  normaliser and entropy, and its most likely outcomes
``score_grad``    the gradient of the log probabilities and the entropy
``distill``       cross-entropy distance (KL) of the row from a teacher that
                  is known by its top logits
``distill_grad``  the gradient of that loss, from the saved log normaliser
``distill_step``  loss and gradient in one call, as a training step makes it

Definitions (c = scale, rows of ``cols`` entries).  The logit of an entry is
the real entry itself, or ln w with w = re^2 + im^2 (each operation rounded
to 32 bits) for an amplitude.  An entry is absent where the mask is zero or
the logit is -inf.  log p = c z - ln sum exp(c z) over the present entries;
the alternatives are the present entries of largest logit (of largest w for
amplitudes), ties to the lowest index, (-1, -inf) past their number.  A row
without present entries has log Z = -inf, entropy 0, loss 0 and no gradient.
A given outcome of -1 has log p = 0; an absent one has -inf and no gradient.
The teacher's probabilities are the softmax of its logits over those of its
outcomes that the row's mask leaves in.
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"c64": torch.complex64, "f32": torch.float32, "bf16": torch.bfloat16,
          "f16": torch.float16}
_BYTES = {"c64": 8, "f32": 4, "bf16": 2, "f16": 2}


def _case(name, op, type_, rows, cols, given=0, top=0, teacher=0, mask=False, scale=1.0):
    return {"name": name, "op": op, "type": type_, "rows": rows, "cols": cols, "given": given,
            "top": top, "teacher": teacher, "mask": mask, "scale": scale}


def listed():
    return [
        # one new token of one sequence: its log probability and a short list
        # of alternatives; all latency
        _case("score_one_token", "score", "bf16", 1, 32768, given=1, top=5),
        # a decoding batch over a large vocabulary, alternatives for sampling
        _case("score_decode_batch", "score", "bf16", 64, 131072, given=1, top=20, scale=1.25),
        # scoring a prompt: many rows, an odd vocabulary (rows not aligned)
        _case("score_prompt_odd", "score", "bf16", 2048, 50001, given=1, top=1),
        # rows post-selected by a mask (a conserved quantity, a grammar)
        _case("score_masked", "score", "f32", 300, 65536, given=4, top=64, mask=True),
        # the amplitudes over 26 open qubits in one row: heavy outcomes, entropy
        _case("score_state", "score", "c64", 1, 1 << 26, given=128, top=100),
        # batches of 64 amplitudes (six open qubits) for many projections
        _case("score_six_qubits", "score", "c64", 20000, 64, given=1, top=4),
        # policy gradient with an entropy bonus over an odd vocabulary
        _case("score_grad_odd", "score_grad", "bf16", 1024, 50001, given=1),
        # likelihood training of a circuit on samples: gradient of 2^20
        # amplitudes
        _case("score_grad_state", "score_grad", "c64", 1, 1 << 20, given=100),
        # a student's training step on a teacher's 32 best tokens
        _case("distill_step_large", "distill_step", "bf16", 1024, 131072, teacher=32, scale=0.5),
        # the same at a smaller vocabulary in 32 bits with masked rows
        _case("distill_step_masked", "distill_step", "f32", 500, 32003, teacher=100, mask=True),
        # a shallow circuit trained on the heavy outcomes of a deep one
        _case("distill_step_circuit", "distill_step", "c64", 16, 16384, teacher=64),
        # the loss alone, for a few evaluation rows
        _case("distill_eval", "distill", "f16", 8, 40000, teacher=8, scale=0.5),
    ]


_MOST_BYTES = 1 << 29       # rows * cols * bytes of the largest listed case's data


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(max(v, lo), hi)


def draw(rng):
    op = rng.choice(["score", "score", "score", "score_grad", "distill", "distill_grad",
                     "distill_step", "distill_step"])
    type_ = rng.choice(["bf16", "bf16", "f16", "f32", "c64"])
    if rng.random() < 0.2:      # few outcomes, many rows
        cols = _log_int(rng, 1, 2048)
        rows = _log_int(rng, 1, 100000)
    elif rng.random() < 0.3:    # long rows, few of them
        cols = _log_int(rng, 1 << 17, 1 << 25)
        rows = _log_int(rng, 1, 16)
    else:
        cols = _log_int(rng, 2048, 1 << 18)
        rows = _log_int(rng, 1, 4096)
    if rng.random() < 0.5:      # aligned rows in one half of the draws
        cols = max(16, cols // 16 * 16)
    writes = 1 if op in ("score", "distill") else 2
    rows = max(1, min(rows, _MOST_BYTES // (cols * _BYTES[type_] * writes)))
    # keep the plain form's 64-bit sort keys within the same bound
    rows = max(1, min(rows, (1 << 27) // cols))
    return {"op": op, "type": type_, "rows": rows, "cols": cols,
            "given": rng.choice([0, 1, 1, 3, 100]) if op == "score"
            else (rng.choice([1, 1, 2, 50]) if op == "score_grad" else 0),
            "top": rng.choice([0, 1, 5, 20, 50, 128]) if op == "score" else 0,
            "teacher": rng.choice([1, 8, 20, 64, 256]) if op.startswith("distill") else 0,
            "mask": rng.random() < 0.3, "scale": rng.choice([1.0, 1.0, 0.5, 1.25])}


# ---- inputs -----------------------------------------------------------------

def _rand_ids(gen, rows, n, cols):
    """Ids as programs have them: mostly in range, some -1 (no token)."""
    ids = torch.randint(0, cols, (rows, n), generator=gen, device="cuda")
    none = torch.rand((rows, n), generator=gen, device="cuda") < 0.03
    return torch.where(none, torch.full_like(ids, -1), ids)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 17)
    R, V, t = case["rows"], case["cols"], case["type"]
    f = {}
    if t == "c64":
        # a random circuit's amplitudes with ten more qubits projected: complex
        # normal, sum |a|^2 about 2^-10
        f["rows"] = torch.view_as_complex(
            torch.randn((R, V, 2), generator=gen, device="cuda") * (0.5 / V / 1024) ** 0.5)
    else:
        # logits of a trained head: a broad normal body and each row its own
        # sharpness
        z = torch.randn((R, V), generator=gen, device="cuda")
        z = z * (1.0 + 2.0 * torch.rand((R, 1), generator=gen, device="cuda"))
        f["rows"] = z.to(_TYPES[t])
        del z
    f["mask"] = None
    if case["mask"]:
        keep = torch.rand((R, 1), generator=gen, device="cuda")
        mask = torch.rand((R, V), generator=gen, device="cuda") < keep
        if R >= 8:
            mask[R // 2] = False          # a row that the mask leaves empty
        f["mask"] = mask
        # what lies in masked places is left over from elsewhere
        bad = torch.rand((R, V), generator=gen, device="cuda") < 0.01
        f["rows"][bad & ~mask] = float("nan")
        f["rows"][~bad & ~mask] = torch.finfo(_TYPES[t]).min if t != "c64" else 0.0
        del bad
    if case["given"]:
        f["given"] = _rand_ids(gen, R, case["given"], V)
    else:
        f["given"] = None
    if case["op"] == "score_grad":
        f["g_logp"] = torch.randn((R, case["given"]), generator=gen, device="cuda") / R
        f["g_entropy"] = torch.randn((R,), generator=gen, device="cuda") * (0.01 / R)
    K = case["teacher"]
    if K:
        ids = _rand_ids(gen, R, K, V)
        logits = torch.sort(torch.randn((R, K), generator=gen, device="cuda") * 2.0,
                            dim=1, descending=True).values
        f["ids"], f["logits"] = ids, logits.contiguous()
        if case["op"] != "distill":
            f["weight"] = torch.rand((R,), generator=gen, device="cuda") / R
    return f


def prepare(case, seed):
    f = _inputs(case, seed)
    f["case"] = dict(case)
    if case["op"] in ("score_grad", "distill_grad"):
        # saved by the forward pass
        _, _, _, logz, entropy = _plain_rows(f["rows"], f["mask"], case["scale"])
        f["logz"] = logz.contiguous()
        f["entropy"] = entropy.contiguous()
    if own:
        import exact_tensor_network_gb300 as tn
        f["op"] = tn.Outcomes(case["cols"], _TYPES[case["type"]], max_rows=case["rows"],
                              top=case["top"], scale=case["scale"])
        f["op"].bind_workspace()
    return f


# ---- the plain form ---------------------------------------------------------

_NEG = float("-inf")


def _plain_order(rows):
    """(order value, logit) of every entry in 32 bits."""
    if rows.is_complex():
        re, im = rows.real, rows.imag
        w = re * re + im * im
        return w, torch.log(w)
    z = rows.float() + 0.0
    return z, z


def _plain_rows(rows, mask, scale):
    """order value, present, scaled logit, log Z and entropy."""
    order, z = _plain_order(rows)
    present = z != _NEG
    if mask is not None:
        present = present & mask
    x = torch.where(present, z * scale, _NEG)
    m = x.amax(dim=1, keepdim=True)
    m = torch.where(m == _NEG, 0.0, m)
    e = torch.exp(x - m)
    logz = m + torch.log(e.sum(dim=1, keepdim=True))
    lp = torch.where(present, x - logz, 0.0)
    entropy = -(torch.exp(lp) * lp * present).sum(dim=1)
    # a row without a distribution (NaN or +inf among its entries)
    entropy = torch.where(torch.isnan(logz[:, 0]), logz[:, 0], entropy)
    return order, present, x, logz[:, 0], entropy


def _plain_given(x, present, logz, ids):
    """log p of the given ids and which of them are present."""
    safe = ids.clamp(min=0)
    here = present.gather(1, safe) & (ids >= 0)
    lp = torch.where(here, x.gather(1, safe) - logz[:, None], _NEG)
    return torch.where(ids < 0, 0.0, lp), here


def _plain_score(s):
    c = s["case"]
    order, present, x, logz, entropy = _plain_rows(s["rows"], s["mask"], c["scale"])
    out = {"logz": logz, "entropy": entropy}
    if c["given"]:
        out["logp"] = _plain_given(x, present, logz, s["given"])[0]
    k = c["top"]
    if k:
        V = c["cols"]
        bits = order.contiguous().view(torch.int32)
        bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
        lowest = torch.iinfo(torch.int64).min
        key = (bits << 32) | (V - 1 - torch.arange(V, device=bits.device))
        key = torch.where(present, key, lowest)
        best = torch.topk(key, min(k, V), dim=1).values
        none = (best == lowest) | torch.isnan(logz[:, None])
        ids = torch.where(none, -1, V - 1 - (best & 0xFFFFFFFF))
        lp = torch.where(none, _NEG, x.gather(1, ids.clamp(min=0)) - logz[:, None])
        lp = torch.where(torch.isnan(logz[:, None]), logz[:, None], lp)
        if k > V:
            ids = torch.nn.functional.pad(ids, (0, k - V), value=-1)
            lp = torch.nn.functional.pad(lp, (0, k - V), value=_NEG)
        out["top_ids"], out["top_logp"] = ids, lp
    return out


def _plain_to_rows(rows, present, gz):
    """The gradient of the logits as one of the rows, rounded once."""
    if rows.is_complex():
        w = rows.real * rows.real + rows.imag * rows.imag
        gz = torch.where(present, 2.0 * gz / w, 0.0)
        return torch.complex(rows.real * gz, rows.imag * gz)
    return torch.where(present, gz, 0.0).to(rows.dtype)


def _plain_score_grad(s):
    c = s["case"]
    order, z = _plain_order(s["rows"])
    present = z != _NEG
    if s["mask"] is not None:
        present = present & s["mask"]
    lp = torch.where(present, z * c["scale"] - s["logz"][:, None], 0.0)
    ids = s["given"]
    safe = ids.clamp(min=0)
    g = torch.where(present.gather(1, safe) & (ids >= 0), s["g_logp"], 0.0)
    gz = -torch.exp(lp) * (g.sum(dim=1, keepdim=True)
                           + s["g_entropy"][:, None] * (lp + s["entropy"][:, None]))
    gz = gz.scatter_add(1, safe, g) * c["scale"]
    return _plain_to_rows(s["rows"], present, gz)


def _plain_teacher(s, present_by_mask):
    """q and log q over the teacher's outcomes that stay in."""
    ids = s["ids"]
    safe = ids.clamp(min=0)
    used = (ids >= 0) & (s["logits"] != _NEG)
    if present_by_mask is not None:
        used = used & present_by_mask.gather(1, safe)
    t = torch.where(used, s["logits"], _NEG)
    m = t.amax(dim=1, keepdim=True)
    m = torch.where(m == _NEG, 0.0, m)
    e = torch.exp(t - m)
    total = e.sum(dim=1, keepdim=True)
    q = torch.where(used, e / total, 0.0)
    logq = torch.where(used, t - m - torch.log(total), 0.0)
    return safe, used, q, logq


def _plain_distill(s):
    c = s["case"]
    order, present, x, logz, _ = _plain_rows(s["rows"], s["mask"], c["scale"])
    safe, used, q, logq = _plain_teacher(s, s["mask"])
    lp = x.gather(1, safe) - logz[:, None]
    loss = torch.where(used & (q > 0), q * (logq - lp), 0.0).sum(dim=1)
    loss = torch.where(logz == _NEG, 0.0, loss)
    return present, x, logz, safe, q, loss


def _plain_distill_gz(s, present, x, logz, safe, q):
    c = s["case"]
    p = torch.exp(torch.where(present, x - logz[:, None], _NEG))
    gz = (p * (q.sum(dim=1, keepdim=True) > 0)).scatter_add(1, safe, -q)
    return _plain_to_rows(s["rows"], present, gz * (s["weight"] * c["scale"])[:, None])


def _plain(s):
    op = s["case"]["op"]
    if op == "score":
        return _plain_score(s)
    if op == "score_grad":
        return {"grad": _plain_score_grad(s)}
    if op == "distill":
        _, _, logz, _, _, loss = _plain_distill(s)
        return {"loss": loss, "logz": logz}
    if op == "distill_grad":
        order, z = _plain_order(s["rows"])
        present = z != _NEG
        if s["mask"] is not None:
            present = present & s["mask"]
        safe, used, q, _ = _plain_teacher(s, s["mask"])
        return {"grad": _plain_distill_gz(s, present, z * s["case"]["scale"], s["logz"], safe, q)}
    present, x, logz, safe, q, loss = _plain_distill(s)
    return {"loss": loss, "logz": logz, "grad": _plain_distill_gz(s, present, x, logz, safe, q)}


# ---- one pass ---------------------------------------------------------------

def run(s):
    if not own:
        return _plain(s)
    op, case = s["op"], s["case"]["op"]
    if case == "score":
        r = op.score(s["rows"], s["given"], mask=s["mask"])
        out = {"logz": r.logz, "entropy": r.entropy}
        if s["given"] is not None:
            out["logp"] = r.logp
        if s["case"]["top"]:
            out["top_ids"], out["top_logp"] = r.top_ids, r.top_logp
        return out
    if case == "score_grad":
        return {"grad": op.score_grad(s["rows"], s["given"], s["logz"], s["entropy"], s["g_logp"],
                                      s["g_entropy"], mask=s["mask"])}
    if case == "distill":
        r = op.distill(s["rows"], s["ids"], s["logits"], mask=s["mask"])
        return {"loss": r.loss, "logz": r.logz}
    if case == "distill_grad":
        return {"grad": op.distill_grad(s["rows"], s["ids"], s["logits"], s["logz"], s["weight"],
                                        mask=s["mask"])}
    r = op.distill_step(s["rows"], s["ids"], s["logits"], s["weight"], mask=s["mask"])
    return {"loss": r.loss, "logz": r.logz, "grad": r.grad}


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    R, V = case["rows"], case["cols"]
    n, b = R * V, _BYTES[case["type"]]
    read = n * b + (n if case["mask"] else 0) + R * case["given"] * 8 + R * case["teacher"] * 12
    op = case["op"]
    if op == "score":
        moved = read + R * (8 + 4 * case["given"] + 12 * case["top"])
        per = 6
    elif op == "score_grad":
        moved = read + R * (4 * case["given"] + 12) + n * b
        per = 7
    elif op == "distill":
        moved = read + 8 * R
        per = 4
    elif op == "distill_grad":
        moved = read + 8 * R + n * b
        per = 5
    else:
        moved = read + 12 * R + n * b
        per = 8
    if case["type"] == "c64":
        per += 5
    return {"bytes": moved, "flops": per * n}


# ---- the definition in 64 bits ----------------------------------------------

def _exact_block(case, f, lo, hi):
    """Rows lo..hi of the definition, in float64; a dict of numpy arrays."""
    def cut(name):
        v = f.get(name)
        return None if v is None else v[lo:hi]
    rows, c, V = cut("rows"), case["scale"], case["cols"]
    inf = float("inf")
    if rows.is_complex():
        a = rows.to(torch.complex128)
        # the order is defined by the weight in 32 bits
        re, im = rows.real.contiguous(), rows.imag.contiguous()
        rank_by = torch.add(re.square(), im.square()).double()
        z = (a.real.square() + a.imag.square()).log()
    else:
        rank_by = z = rows.double()
    keep = torch.ones_like(z, dtype=torch.bool) if f["mask"] is None else cut("mask")
    out = keep.logical_not() | z.isneginf()
    y = (c * z).masked_fill(out, -inf)
    logz = torch.logsumexp(y, dim=1)
    empty = out.all(dim=1)
    op = case["op"]
    logp = (y - logz[:, None])
    logp[empty] = -inf
    p = logp.exp()
    result = {}
    if op in ("score", "score_grad"):
        entropy = torch.special.entr(p).sum(dim=1)
        ids = cut("given")
        if ids is not None:
            pick = ids.clamp(min=0)
            absent = out.gather(1, pick)
    if op == "score":
        result["logz"], result["entropy"] = logz, entropy
        if ids is not None:
            result["logp"] = logp.gather(1, pick).masked_fill(ids < 0, 0.0)
        k = case["top"]
        if k:
            by = rank_by.masked_fill(out, -inf)
            ids_all = torch.sort(by, dim=1, descending=True, stable=True).indices[:, :k]
            gone = out.gather(1, ids_all)
            tl = logp.gather(1, ids_all)
            top_ids = torch.full((hi - lo, k), -1, dtype=torch.int64, device=rows.device)
            top_lp = torch.full((hi - lo, k), -inf, dtype=torch.float64, device=rows.device)
            top_ids[:, :ids_all.shape[1]] = ids_all.masked_fill(gone, -1)
            top_lp[:, :ids_all.shape[1]] = tl.masked_fill(gone, -inf)
            result["top_ids"], result["top_logp"] = top_ids, top_lp
        return result
    if op == "score_grad":
        g = cut("g_logp").double().masked_fill(absent | (ids < 0), 0.0)
        inner = g.sum(dim=1, keepdim=True) + cut("g_entropy").double()[:, None] * (
            logp.masked_fill(out, 0.0) + entropy[:, None])
        gz = -(p * inner)
        gz.scatter_add_(1, pick, g)
        gz *= c
    else:
        ids, t = cut("ids"), cut("logits").double()
        pick = ids.clamp(min=0)
        t = t.masked_fill((ids < 0) | keep.gather(1, pick).logical_not(), -inf)
        none = t.isneginf().all(dim=1)
        q = torch.softmax(t, dim=1)
        q[none] = 0.0
        lp_at = logp.gather(1, pick)
        loss = (torch.xlogy(q, q) - torch.where(q > 0, q * lp_at, 0.0)).sum(dim=1)
        loss[empty] = 0.0
        if op != "distill_grad":
            result["loss"], result["logz"] = loss, logz
        if op == "distill":
            return result
        gz = p.clone()
        gz[none] = 0.0
        gz.scatter_add_(1, pick, -q)
        gz *= c * cut("weight").double()[:, None]
    gz = gz.masked_fill(out, 0.0)
    if rows.is_complex():
        a2 = a.real.square() + a.imag.square()
        result["grad"] = torch.where(out, 0.0, 2.0 * gz / a2) * a
    else:
        result["grad"] = gz
    return result


def exact(case, seed):
    f = _inputs(case, seed)
    R, V = case["rows"], case["cols"]
    step = max(1, (1 << 24) // V)
    parts = []
    for lo in range(0, R, step):
        block = _exact_block(case, f, lo, min(R, lo + step))
        parts.append({k: v.cpu().numpy() for k, v in block.items()})
    return {k: np.concatenate([p[k] for p in parts]) for k in parts[0]}
