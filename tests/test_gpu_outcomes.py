"""Outcome operators against their definitions in 64 bits.

Tolerances (derived, u = 2^-24 the fp32 rounding):
* log Z: every exponential carries the exponential unit's error (2 ulp = 4 u),
  its argument's roundings (3 u |d|, whose weighted mean is at most the
  entropy plus the reference's lag of 8 powers of two), sums of at most a few
  hundred sequential terms of random-signed roundings (8 u), and the final sum
  rounds |scale z| and |log Z|.  In all below 16 u (1 + M + H), M = max |scale z|.
* log p adds one rounding of each; entropy the same error once more (ln s - t / s).
* gradients: p inherits log p's absolute error as a relative one; the result
  is rounded to the rows' type once.
Ids have to be equal."""
import numpy as np
import pytest

import exact_tensor_network_gb300 as tn
from outcome_reference import INF, Row

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
OUT_EPS = {"f32": 2 * U, "bf16": 2.0 ** -8, "f16": 2.0 ** -11, "c64": 8 * U}
# smallest steps of the types: results below underflow
OUT_MIN = {"f32": 1e-44, "bf16": 1e-40, "f16": 2.0 ** -24, "c64": 1e-44}
TYPES = ["c64", "f32", "bf16", "f16"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


def torch_type(t):
    import torch
    return {"c64": torch.complex64, "f32": torch.float32, "bf16": torch.bfloat16,
            "f16": torch.float16}[t]


def make_rows(rng, R, V, t, spread=3.0):
    import torch
    if t == "c64":
        a = (rng.standard_normal((R, V)) + 1j * rng.standard_normal((R, V))) / np.sqrt(2.0 * V)
        return torch.from_numpy(a.astype(np.complex64))
    z = torch.from_numpy((spread * rng.standard_normal((R, V))).astype(np.float32))
    return z.to(torch_type(t))


def to_np(x):
    import torch
    if x.dtype in (torch.bfloat16, torch.float16):
        x = x.float()
    return x.cpu().numpy()


def close(got, ref, tol, what):
    got, ref = np.asarray(got, dtype=ref.dtype), np.asarray(ref)
    tol = np.broadcast_to(tol, ref.shape)
    nan = np.isnan(ref)
    assert (np.isnan(got) == nan).all(), f"{what}: NaN in other places"
    inf = np.isinf(ref) if not np.iscomplexobj(ref) else np.zeros(ref.shape, bool)
    assert (got[inf] == ref[inf]).all(), f"{what}: infinities differ"
    ok = ~(nan | inf)
    err = np.abs(got[ok] - ref[ok])
    worst = (err - tol[ok]).max() if err.size else -1.0
    assert worst <= 0, (f"{what}: error {err[np.argmax(err - tol[ok])]:.3e} above its bound "
                        f"{tol[ok][np.argmax(err - tol[ok])]:.3e}")


def tol_logz(r):
    return 16 * U * (1 + r.mag + abs(r.entropy if np.isfinite(r.entropy) else 0.0))


def run_all(rows, t, given, top, teacher, mask=None, scale=1.0, grad_out=None, max_rows=None,
            teacher_scale=1.0, teacher_type="f32", rng=None):
    """Every call on these rows (a CPU tensor or a CUDA view) against the
    definitions."""
    import torch
    rng = rng or np.random.default_rng(1)
    d_rows = rows if rows.is_cuda else rows.cuda()
    R, V = d_rows.shape
    d_mask = None if mask is None else (mask if mask.is_cuda else mask.cuda())
    op = tn.Outcomes(V, torch_type(t), max_rows=max_rows or R, top=top, scale=scale)
    h_rows = to_np(d_rows)
    h_mask = None if mask is None else np.broadcast_to(to_np(d_mask), (R, V))
    ref = [Row(h_rows[i], None if h_mask is None else h_mask[i], scale) for i in range(R)]
    d_given = None if given is None else torch.from_numpy(given).cuda()
    s = op.score(d_rows, d_given, mask=d_mask)
    torch.cuda.synchronize()
    op.check()
    tz = np.array([tol_logz(r) for r in ref])
    close(to_np(s.logz), np.array([r.logz for r in ref]), tz, "log Z")
    close(to_np(s.entropy), np.array([r.entropy for r in ref]), 2 * tz, "entropy")
    if given is not None:
        want = np.stack([r.logp(given[i].reshape(-1)) for i, r in enumerate(ref)])
        close(to_np(s.logp).reshape(R, -1), want, 2 * tz[:, None], "log p")
    if top:
        want = [r.top(top) for r in ref]
        assert (to_np(s.top_ids) == np.stack([w[0] for w in want])).all(), "alternatives differ"
        close(to_np(s.top_logp), np.stack([w[1] for w in want]), 2 * tz[:, None], "alternatives' log p")

    def close_grad(got, pairs, what):
        want = np.stack([p[0] for p in pairs])
        scale_ = np.stack([p[1] for p in pairs])
        size = np.abs(np.where(np.isnan(want), 0, want))
        # log p's error, p's own units, and the rounding to the type
        tol = (4 * tz[:, None] + 16 * U) * scale_ + OUT_EPS[t] * size + OUT_MIN[t]
        close(to_np(got), want, tol, what)

    if given is not None:
        n = given.reshape(R, -1).shape[1]
        g = rng.standard_normal((R, n)).astype(np.float32)
        h = rng.standard_normal(R).astype(np.float32)
        d_g = torch.from_numpy(g).reshape(given.shape).cuda()
        d_h = torch.from_numpy(h).cuda()
        got = op.score_grad(d_rows, d_given, s.logz, s.entropy, d_g, d_h, mask=d_mask, out=grad_out)
        close_grad(got, [r.score_grad(given[i].reshape(-1), g[i], h[i]) for i, r in enumerate(ref)],
                   "score gradient")
        got = op.score_grad(d_rows, d_given, s.logz, s.entropy, d_g, mask=d_mask, out=grad_out)
        close_grad(got, [r.score_grad(given[i].reshape(-1), g[i]) for i, r in enumerate(ref)],
                   "score gradient without entropy")
    if teacher is not None:
        ids, logits = teacher
        lt = torch.from_numpy(logits).to(torch_type(teacher_type))
        lref = to_np(lt).astype(np.float64) * np.float64(np.float32(teacher_scale))
        d_ids, d_l = torch.from_numpy(ids).cuda(), lt.cuda()
        w = rng.standard_normal(R).astype(np.float32)
        d_w = torch.from_numpy(w).cuda()
        r1 = op.distill(d_rows, d_ids, d_l, mask=d_mask, teacher_scale=teacher_scale)
        r2 = op.distill_step(d_rows, d_ids, d_l, d_w, mask=d_mask, teacher_scale=teacher_scale,
                             out=grad_out)
        close_grad(r2.grad, [r.distill_grad(ids[i], lref[i], w[i]) for i, r in enumerate(ref)],
                   "distill step gradient")
        g2 = op.distill_grad(d_rows, d_ids, d_l, r1.logz, d_w, mask=d_mask,
                             teacher_scale=teacher_scale, out=grad_out)
        close_grad(g2, [r.distill_grad(ids[i], lref[i], w[i]) for i, r in enumerate(ref)],
                   "distill gradient")
        want = np.array([r.distill(ids[i], lref[i]) for i, r in enumerate(ref)])
        fin = np.where(np.isfinite(lref), np.abs(lref), 0.0)
        tl = 2 * tz + 16 * U * (1 + fin.max(axis=1))
        for what, r in (("distill", r1), ("distill step", r2)):
            close(to_np(r.loss), want, tl, what + " loss")
            close(to_np(r.logz), np.array([x.logz for x in ref]), tz, what + " log Z")
        torch.cuda.synchronize()
        op.check()
    return op


def rand_ids(rng, R, n, V):
    ids = rng.integers(0, V, size=(R, n))
    ids[rng.random((R, n)) < 0.1] = -1
    return ids.astype(np.int64)


def rand_teacher(rng, R, K, V):
    t = (2.0 * rng.standard_normal((R, K))).astype(np.float32)
    t[rng.random((R, K)) < 0.05] = -INF
    return rand_ids(rng, R, K, V), t


SHAPES = [(1, 1), (5, 1), (3, 2), (7, 7), (2, 31), (33, 64), (9, 255), (4, 1000), (3, 2049), (2, 4099),
          (5, 8192), (1, 50001), (3, 50000), (1, 300007)]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_matches_definition(shape, t):
    R, V = shape
    rng = np.random.default_rng(R * 1000003 + V)
    run_all(make_rows(rng, R, V, t), t, rand_ids(rng, R, 3, V), 5, rand_teacher(rng, R, 9, V), rng=rng)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("scale", [0.125, 0.7, 2.5])
@pytest.mark.parametrize("shape", [(6, 333), (2, 20011)], ids=lambda s: f"{s[0]}x{s[1]}")
def test_temperatures(shape, scale, t):
    R, V = shape
    rng = np.random.default_rng(V)
    run_all(make_rows(rng, R, V, t), t, rand_ids(rng, R, 2, V), 4, rand_teacher(rng, R, 20, V),
            scale=scale, teacher_scale=scale, teacher_type="bf16" if t == "bf16" else "f16", rng=rng)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("shape", [(12, 77), (10, 1601), (9, 9001), (3, 65537)],
                         ids=lambda s: f"{s[0]}x{s[1]}")
@pytest.mark.parametrize("kind", ["random", "prefix", "one_row", "one_column"])
def test_masks(shape, kind, t):
    """Masked rows, an empty one among them; NaN, infinities and the type's
    lowest value lie in masked places."""
    import torch
    R, V = shape
    rng = np.random.default_rng(V + len(kind))
    rows = make_rows(rng, R, V, t)
    if kind == "random":
        keep = rng.random((R, V)) < rng.random((R, 1))
        keep[R // 2] = False
    elif kind == "prefix":
        keep = np.arange(V)[None, :] < rng.integers(0, V + 1, size=(R, 1))
        keep[0] = False
        keep[1] = np.arange(V) < 1
    elif kind == "one_row":
        keep = rng.random((1, V)) < 0.5
    else:
        keep = rng.random((R, 1)) < 0.5
        keep[0], keep[1] = True, False
    mask = torch.from_numpy(keep)
    out = ~np.broadcast_to(keep, (R, V))
    junk = rng.integers(0, 4, size=(R, V))
    for v, x in enumerate([float("nan"), INF, -INF, float(torch.finfo(torch_type(t)).min)]):
        rows[torch.from_numpy(out & (junk == v))] = x
    run_all(rows, t, rand_ids(rng, R, 4, V), 7, rand_teacher(rng, R, 30, V), mask=mask, rng=rng)


def _views(t, kind):
    """(rows, mask, grad out) views of one layout, 5 x 3001."""
    import torch
    rng = np.random.default_rng(11)
    R, V = 5, 3001
    data = make_rows(rng, R, V, t).cuda()
    keep = torch.from_numpy(rng.random((R, V)) < 0.7).cuda()

    def place(x):
        if kind == "padded":
            buf = torch.zeros((R, V + 13), dtype=x.dtype, device="cuda")
            v = buf[:, 5:5 + V]
        elif kind == "every_second":
            v = torch.zeros((R, 2 * V), dtype=x.dtype, device="cuda")[:, ::2]
        elif kind == "transposed":
            v = torch.zeros((V, R), dtype=x.dtype, device="cuda").t()
        else:   # rows far apart, first one odd
            buf = torch.zeros((R * 2, V + 1), dtype=x.dtype, device="cuda")
            v = buf[1::2, 1:]
        v.copy_(x)
        return v
    return place(data), place(keep), place(torch.zeros_like(data)), rng


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("kind", ["padded", "every_second", "transposed", "far"])
@pytest.mark.parametrize("masked", [False, True])
def test_strides(kind, masked, t):
    rows, keep, out, rng = _views(t, kind)
    R, V = rows.shape
    run_all(rows, t, rand_ids(rng, R, 3, V), 6, rand_teacher(rng, R, 11, V),
            mask=keep if masked else None, grad_out=out, rng=rng)
    # the same with a contiguous gradient, whose alignment differs
    run_all(rows, t, rand_ids(rng, R, 3, V), 6, rand_teacher(rng, R, 11, V),
            mask=keep if masked else None, rng=rng)


def test_repeated_row_view():
    """Row stride 0 (an expanded row)."""
    rng = np.random.default_rng(5)
    row = make_rows(rng, 1, 777, "f32").cuda()
    run_all(row.expand(6, 777), "f32", rand_ids(rng, 6, 2, 777), 3, rand_teacher(rng, 6, 4, 777), rng=rng)


@pytest.mark.parametrize("k", [1, 2, 33, 128])
@pytest.mark.parametrize("order", ["ascending", "descending", "equal", "two_values", "few", "zeros",
                                   "block"])
@pytest.mark.parametrize("shape", [(3, 100), (3, 1700), (2, 30000), (4, 262144), (1, 1500001)],
                         ids=lambda s: f"{s[0]}x{s[1]}")
def test_alternatives_of_hard_rows(shape, order, k):
    """Sorted rows, ties everywhere (lowest index first), fewer present
    entries than alternatives, signed zeros, all the best side by side."""
    import torch
    R, V = shape
    rng = np.random.default_rng(k)
    z = np.zeros((R, V), np.float32)
    if order == "ascending":
        z[:] = np.arange(V) * (30.0 / V)
    elif order == "descending":
        z[:] = -np.arange(V) * (30.0 / V)
    elif order == "equal":
        z[:] = 1.5
    elif order == "two_values":
        z[:] = rng.integers(0, 2, size=(R, V))
    elif order == "few":
        z[:] = -INF
        for r in range(R):
            z[r, rng.integers(0, V, size=5)] = rng.standard_normal(5)
    elif order == "zeros":
        z[:] = np.where(rng.random((R, V)) < 0.5, 0.0, -0.0)
    else:
        z[:] = rng.standard_normal((R, V))
        z[:, V // 3:V // 3 + 200] += 20.0
    for t in ("f32", "bf16"):
        run_all(torch.from_numpy(z).to(torch_type(t)), t, None, k, None)


@pytest.mark.parametrize("t", ["bf16", "c64"])
def test_many_rows_of_one_cta_each(t):
    """Rows that fill the GPU alone: one segment per row, maxima of 32
    vectors."""
    V = {"bf16": 20001, "c64": 2501}[t]
    rng = np.random.default_rng(3)
    run_all(make_rows(rng, 640, V, t), t, rand_ids(rng, 640, 1, V), 20, None, rng=rng)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("scale", [1.0, 0.7])
@pytest.mark.parametrize("V", [1, 60, 5000, 200000])
def test_only_entry_is_certain(V, scale, t):
    """One entry present: log p and entropy are exactly 0, and so are the
    gradients, whatever the entry's value."""
    import torch
    rng = np.random.default_rng(V)
    R = 40
    at = rng.integers(0, V, size=(R, 1))
    z = np.zeros((R, V), np.complex64) if t == "c64" else np.full((R, V), -INF, np.float32)
    np.put_along_axis(z, at, (rng.standard_normal((R, 1)) * 5 + 0.1).astype(z.dtype), axis=1)
    rows = torch.from_numpy(z).to(torch_type(t)).cuda()
    ids = torch.from_numpy(at).cuda()
    op = tn.Outcomes(V, torch_type(t), max_rows=R, top=2, scale=scale)
    s = op.score(rows, ids)
    g = op.score_grad(rows, ids, s.logz, s.entropy, torch.ones((R, 1), device="cuda"),
                      torch.ones(R, device="cuda"))
    d = op.distill_step(rows, ids, torch.ones((R, 1), device="cuda"), torch.ones(R, device="cuda"))
    op.check()
    for x in (s.entropy, s.logp, s.top_logp[:, 0], g, d.loss, d.grad):
        assert (x == 0).all()
    assert (s.top_ids[:, :1] == ids).all() and (s.top_ids[:, 1] == -1).all()


@pytest.mark.parametrize("k", [3, 100])
@pytest.mark.parametrize("order", ["random", "equal", "few", "masked", "block"])
@pytest.mark.parametrize("t", ["c64", "bf16"])
def test_alternatives_of_very_long_rows(t, order, k):
    """Rows whose pieces' maxima form a tree: every outcome as likely as the
    next, a handful of outcomes, the best ones side by side."""
    import torch
    R, V = 2, 2500003
    rng = np.random.default_rng(k)
    rows, mask = make_rows(rng, R, V, t), None
    if order == "equal":
        rows[:] = 0.25
    elif order == "few":
        keep = torch.zeros((R, V), dtype=torch.bool)
        for r in range(R):
            keep[r, torch.from_numpy(rng.integers(0, V, size=50))] = True
        rows[~keep] = 0.0 if t == "c64" else -INF
    elif order == "masked":
        mask = torch.from_numpy(rng.random((1, V)) < 0.3)
    elif order == "block":
        rows[:, V // 2:V // 2 + 300] *= 64.0
    run_all(rows, t, rand_ids(rng, R, 2, V), k, None, mask=mask, rng=rng)


@pytest.mark.parametrize("t,V,k", [("bf16", 30000001, 3), ("c64", 8000001, 20), ("f32", 16000000, 100)])
def test_search_of_very_long_rows_does_not_vary(t, V, k):
    """Rows with four segments an alternative or more: the search goes down
    its three levels one right after the other.  Every warp has to see every
    level's count before the next level clears it, in each of many calls."""
    import torch
    rows = torch.randn((1, V), generator=torch.Generator().manual_seed(V), dtype=torch.float32)
    if t == "c64":
        rows = torch.complex(rows, rows.flip(1)) * V ** -0.5
    rows = rows.to(torch_type(t)).cuda()
    op = tn.Outcomes(V, torch_type(t), top=k)
    got = [op.score(rows) for _ in range(100)]
    ids, lp = Row(to_np(rows)[0], None, 1.0).top(k)
    for s in got:
        assert (to_np(s.top_ids)[0] == ids).all()
        assert (s.top_logp == got[0].top_logp).all() and (s.logz == got[0].logz).all()


@pytest.mark.parametrize("k", [1, 60, 128])
@pytest.mark.parametrize("t,R,V", [("f32", 40, 300007), ("bf16", 64, 400001), ("c64", 3, 3000001),
                                   ("f32", 700, 40001)])
@pytest.mark.parametrize("part", ["all", "start", "place"])
def test_alternatives_of_a_part(t, R, V, k, part):
    """Long rows in few and in many segments, with entries everywhere, at the
    start only, or at one place only."""
    import torch
    rng = np.random.default_rng(V + k)
    if R * V > 2e7 and part != "all":
        R //= 10
    mask = None
    if part != "all":
        keep = np.zeros((1, V), bool)
        if part == "start":
            keep[0, :V // 20] = True
        else:
            keep[0, V // 2:V // 2 + 900] = True
        mask = torch.from_numpy(keep)
    run_all(make_rows(rng, R, V, t), t, None, k, None, mask=mask, rng=rng)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("t,R,V", [("bf16", 2500, 2601), ("c64", 1300, 1031), ("f32", 700, 5003)])
def test_many_rows(t, R, V, masked):
    """More rows than the GPU holds groups, odd lengths, a mask of its own
    for every row (an empty one among them)."""
    import torch
    rng = np.random.default_rng(V)
    keep = None
    if masked:
        keep = rng.random((R, V)) < rng.random((R, 1))
        keep[R // 3] = False
        keep = torch.from_numpy(keep)
    run_all(make_rows(rng, R, V, t), t, rand_ids(rng, R, 1, V), 3 if masked else 40,
            rand_teacher(rng, R, 17, V), mask=keep, rng=rng)


@pytest.mark.parametrize("k", [1, 50, 128])
@pytest.mark.parametrize("t,R,V", [("f16", 2500, 5003), ("c64", 2500, 901), ("f32", 2500, 4090)])
def test_alternatives_in_a_warp(t, R, V, k):
    """Rows enough for a warp each, whose maxima lie over two or four
    vectors; among them equal, sorted, masked and empty ones."""
    import torch
    rng = np.random.default_rng(V + k)
    rows = make_rows(rng, R, V, t)
    rows[1] = 0.5
    rows[2, 7:] = 0.0 if t == "c64" else -INF
    if t != "c64":
        rows[3] = torch.sort(rows[3].float()).values.to(rows.dtype)
        rows[4] = torch.sort(rows[4].float(), descending=True).values.to(rows.dtype)
    keep = rng.random((R, V)) < 0.9
    keep[5] = False
    keep[6, 30:] = False
    run_all(rows, t, None, k, None, mask=torch.from_numpy(keep), rng=rng)


@pytest.mark.parametrize("t,V", [(t, V) for t, at in (("bf16", 4097), ("f16", 4097), ("f32", 2049), ("c64", 1025))
                                 for V in (at - 7, at - 3, at - 1, at, at + 1, at + 7)])
def test_best_entry_ends_a_warps_row(t, V):
    """Rows of one warp each around the length at which their maxima double in
    size (512 vectors, with and without room for a misaligned start): every
    maximum counts, the one of the row's last vector too."""
    import torch
    R = 2500
    rng = np.random.default_rng(V)
    rows = make_rows(rng, R, V, t)
    rows[::2, V - 1] = 40.0
    rows[::3, V - 2] = 30.0
    run_all(rows, t, None, 3, None, rng=rng)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("t,R,V", [("f16", 4900, 2203), ("c64", 4900, 601), ("f32", 470, 4001)])
def test_warps_hold_longer_rows(t, R, V, masked):
    """Rows enough that a warp each is faster than a CTA each; many of the
    teacher's outcomes are repeated."""
    import torch
    rng = np.random.default_rng(V)
    keep = torch.from_numpy(rng.random((R, V)) < 0.5) if masked else None
    ids, logits = rand_teacher(rng, R, 90, V)
    ids[:, ::2] %= 300
    ids[:, 1::7] = ids[:, :1]
    given = rand_ids(rng, R, 40, V)
    given[:, 1::2] = given[:, ::2]
    run_all(make_rows(rng, R, V, t), t, given, 0, (ids, logits), mask=keep, rng=rng)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("t,R,V", [("bf16", 30, 70001), ("f32", 21, 90001), ("c64", 9, 150001),
                                   ("f16", 3, 900001), ("f32", 2, 800003)])
def test_distillation_of_long_rows(t, R, V, masked):
    """Rows that several CTAs hold between them, and rows too long for that."""
    import torch
    rng = np.random.default_rng(V)
    keep = None
    if masked:
        keep = rng.random((R, V)) < 0.5
        keep[1] = False
        keep[0, :V - 9] = False
        keep = torch.from_numpy(keep)
    run_all(make_rows(rng, R, V, t), t, None, 0, rand_teacher(rng, R, 200, V), mask=keep, rng=rng)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("V", [50, 40000])
def test_rows_without_distribution(V, t):
    """NaN and +inf in present places, -inf everywhere, the lowest value
    everywhere; neighbours are untouched."""
    import torch
    rng = np.random.default_rng(9)
    rows = make_rows(rng, 6, V, t)
    rows[1, V // 2] = float("nan")
    rows[3, V - 1] = INF
    rows[4] = -INF if t != "c64" else 0.0
    if t != "c64":
        rows[5] = -INF
        rows[5, 7] = 2.0        # one outcome left: probability one
    run_all(rows, t, rand_ids(rng, 6, 4, V), 5, rand_teacher(rng, 6, 6, V), rng=rng)
    if t in ("f32", "bf16"):
        low = torch.full((2, V), float(torch.finfo(torch_type(t)).min), dtype=torch_type(t)).cuda()
        s = tn.Outcomes(V, torch_type(t), max_rows=2, top=3).score(low)
        assert (to_np(s.top_ids) == [0, 1, 2]).all()
        np.testing.assert_allclose(to_np(s.entropy), np.log(V), rtol=1e-5)
        np.testing.assert_allclose(to_np(s.logz), float(torch.finfo(torch_type(t)).min), rtol=1e-6)


def _check_filled_rows(t, fill, scale, V, layout):
    """Rows whose unwanted entries hold a large negative logit instead of
    -inf.  Beside ordinary logits its weight is 0, so that everything but the
    fill's own log p is as for -inf, within the bounds of those rows (M is of
    the ordinary logits).  A row of nothing else is uniform."""
    import torch
    rng = np.random.default_rng(V)
    R, K = 5, 6
    rows = make_rows(rng, R, V, t)
    out = rng.random((R, V)) < 0.5
    out[0, :V // 2] = True                  # whole vectors before any ordinary logit
    out[1, V // 2:] = True                  # and after
    out[2, :V - 1] = True
    out[2, V - 1] = False
    out[3] = True
    rows[torch.from_numpy(out)] = fill
    clean = to_np(rows).copy()
    clean[out] = -INF
    buf = torch.zeros((R, 2 * V + 16), dtype=rows.dtype, device="cuda")
    d = {"aligned": buf[:, :V], "misaligned": buf[:, 1:V + 1], "strided": buf[:, ::2][:, :V]}[layout]
    if layout == "aligned":
        d = torch.empty((R, (V + 7) // 8 * 8), dtype=rows.dtype, device="cuda")[:, :V]
    d.copy_(rows)
    ids = np.stack([rng.choice(np.flatnonzero(~out[i]), K) if i != 3 else rng.integers(0, V, K) for i in range(R)])
    logits = rng.standard_normal((R, K)).astype(np.float32)
    w = rng.standard_normal(R).astype(np.float32)
    d_ids, d_l, d_w = torch.from_numpy(ids).cuda(), torch.from_numpy(logits).cuda(), torch.from_numpy(w).cuda()
    op = tn.Outcomes(V, torch_type(t), max_rows=R, top=3, scale=scale)
    s = op.score(d, d_ids)
    ref = [Row(clean[i], None, scale) for i in range(R)]
    tz = np.array([tol_logz(r) for r in ref])
    some = [0, 1, 2, 4]
    close(to_np(s.logz)[some], np.array([ref[i].logz for i in some]), tz[some], "log Z")
    close(to_np(s.entropy)[some], np.array([ref[i].entropy for i in some]), 2 * tz[some], "entropy")
    close(to_np(s.logp)[some], np.stack([ref[i].logp(ids[i]) for i in some]), 2 * tz[some][:, None], "log p")
    for i in some:
        n = min(3, int((~out[i]).sum()))
        assert (to_np(s.top_ids)[i][:n] == ref[i].top(3)[0][:n]).all()
    np.testing.assert_allclose(to_np(s.logz)[3], float(d[3, 0]) * scale, rtol=1e-6)
    np.testing.assert_allclose(to_np(s.entropy)[3], np.log(V), rtol=1e-5)
    assert to_np(s.top_ids)[3].tolist() == [0, 1, 2]
    g = w[:, None] * logits
    got = to_np(op.score_grad(d, d_ids, s.logz, s.entropy, torch.from_numpy(g).cuda()))
    loss = op.distill(d, d_ids, d_l)
    step = op.distill_step(d, d_ids, d_l, d_w)
    dg = to_np(op.distill_grad(d, d_ids, d_l, loss.logz, d_w))
    for what, x in (("distill", loss), ("distill step", step)):
        close(to_np(x.logz)[some], np.array([ref[i].logz for i in some]), tz[some], what + " log Z")
        want = np.array([ref[i].distill(ids[i], logits[i].astype(np.float64)) for i in some])
        close(to_np(x.loss)[some], want, 2 * tz[some] + 64 * U, what + " loss")
    for i in some:
        for what, x, (want, mag) in (
                ("score", got, ref[i].score_grad(ids[i], g[i])),
                ("step", to_np(step.grad), ref[i].distill_grad(ids[i], logits[i].astype(np.float64), w[i])),
                ("distill", dg, ref[i].distill_grad(ids[i], logits[i].astype(np.float64), w[i]))):
            tol = (4 * tz[i] + 16 * U) * mag + OUT_EPS[t] * np.abs(want) + OUT_MIN[t]
            close(x[i], want, tol, what + " gradient")
    # the uniform row: p = 1 / V from the sums (log Z itself rounds to the fill's)
    uniform = Row(np.zeros(V, np.float32), None, scale)
    want, mag = uniform.distill_grad(ids[3], logits[3].astype(np.float64), w[3])
    if V * d.element_size() < 60000:            # the row is held on chip
        dense = np.setdiff1d(np.arange(V), np.concatenate([ids[3], [*range(8), *range(V - 8, V)]]))
        if layout != "strided":
            close(to_np(step.grad)[3][dense], want[dense],
                  (1e-5 * mag + OUT_EPS[t] * np.abs(want) + OUT_MIN[t])[dense], "uniform row's gradient")
    assert np.isfinite(to_np(step.grad)[3]).all() and np.isfinite(got[3]).all()


@pytest.mark.parametrize("layout", ["aligned", "misaligned", "strided"])
@pytest.mark.parametrize("V", [75, 4001, 50001])
@pytest.mark.parametrize("scale", [2.0 ** -40, 0.01, 0.05, 0.08, 0.3, 1.0])
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_lowest_values_at_high_temperature(t, scale, V, layout):
    """The type's lowest value, and one between it and -2^126: c z may be small
    there although z is not."""
    import torch
    _check_filled_rows(t, float(torch.finfo(torch_type(t)).min), scale, V, layout)
    _check_filled_rows(t, -1.2e38, scale, V, layout)


@pytest.mark.parametrize("layout", ["aligned", "misaligned", "strided"])
@pytest.mark.parametrize("V", [75, 4001, 50001])
@pytest.mark.parametrize("scale", [0.08, 0.7, 1.0, 1.25])
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_large_fills(t, scale, V, layout):
    """What masks are written as, from 1e9 to 1e37: scale log2(e) z rounds by
    2^6 and more from 2^30 on."""
    for fill in (-1e9, -2e9, -1e10, -1e12, -1e20, -1e30, -1e37):
        _check_filled_rows(t, fill, scale, V, layout)


@pytest.mark.parametrize("V", [75, 4001, 50001])
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_large_logits(t, V):
    """Logits whose differences are lost beside them, and all of whose
    neighbours are below e^-44 (2^-64): the largest alone is left, wherever it
    stands and whichever ones come before it.  Large scales of ordinary ones
    are the same case."""
    import torch
    rng = np.random.default_rng(V)
    R = 12
    for unit, scale in ((1e9, 2.0), (3e9, 1.0), (1e10, 1.0), (1e20, 0.7), (1e30, 1.25), (3.0, 2.0 ** 30),
                        (3.0, 2.0 ** 40)):
        z = rng.standard_normal((R, V)) * unit
        z[3] = -np.abs(z[3])
        z[4] = np.sort(z[4])
        z[5] = -np.sort(z[5])
        z[6] = -1e9 * (1 + rng.random(V))           # on both sides of 2^30
        z[7] = 1e9 * (1 + rng.random(V))
        rows = torch.from_numpy(z.astype(np.float32)).to(torch_type(t))
        h = to_np(rows).astype(np.float64)
        best = h.max(axis=1)
        many = (h == best[:, None]).sum(axis=1)
        d = rows.cuda()
        ids = torch.from_numpy(h.argmax(axis=1)[:, None]).cuda()
        op = tn.Outcomes(V, torch_type(t), max_rows=R, top=2, scale=scale)
        s = op.score(d, ids)
        x = op.distill(d, ids, torch.zeros((R, 1), device="cuda"))
        step = op.distill_step(d, ids, torch.zeros((R, 1), device="cuda"), torch.ones(R, device="cuda"))
        assert (s.top_ids[:, :1] == ids).all()
        for lz in (s.logz, x.logz, step.logz):
            np.testing.assert_allclose(to_np(lz), best * scale, rtol=4 * U, atol=np.log(V))
        np.testing.assert_allclose(to_np(s.entropy), np.log(many), rtol=1e-5, atol=1e-6)
        got = to_np(step.grad)
        assert np.isfinite(got).all()
        assert (got[h < best[:, None]] == 0).all(), (unit, scale)
        one = many == 1
        assert (got[one, h.argmax(axis=1)[one]] == 0).all()


def _check_amplitudes(rows, scale, rng, grad_floor):
    """Every call on complex64 rows against the definitions, at any scale.

    The bounds are those of the module for log Z (the rounding of scale ln w,
    and so M, is most of it at large scales).  A gradient's p has log p's error
    as an exponent, its factor log p + H has that error once more, and p below
    2^-126 may count as 0 where ``grad_floor``."""
    import torch
    R, V = rows.shape
    K = 6
    d = rows.cuda()
    h_rows = to_np(rows)
    ids = rand_ids(rng, R, K, V)
    with np.errstate(under="ignore"):
        ids[:, 0] = (h_rows.real ** 2 + h_rows.imag ** 2).argmax(axis=1)
    logits = rng.standard_normal((R, K)).astype(np.float32)
    g = rng.standard_normal((R, K)).astype(np.float32)
    h, w = rng.standard_normal(R).astype(np.float32), rng.standard_normal(R).astype(np.float32)
    dev = [torch.from_numpy(x).cuda() for x in (ids, logits, g, h, w)]
    op = tn.Outcomes(V, torch.complex64, max_rows=R, top=4, scale=scale)
    s = op.score(d, dev[0])
    gs = to_np(op.score_grad(d, dev[0], s.logz, s.entropy, dev[2], dev[3]))
    loss = op.distill(d, dev[0], dev[1])
    gd = to_np(op.distill_grad(d, dev[0], dev[1], loss.logz, dev[4]))
    step = op.distill_step(d, dev[0], dev[1], dev[4])
    torch.cuda.synchronize()
    op.check()
    for i in range(R):
        r = Row(h_rows[i], None, scale)
        tz = tol_logz(r)
        top = r.top(4)
        assert (to_np(s.top_ids)[i] == top[0]).all(), "alternatives differ"
        one = np.ones(1)
        for what, got, want, tol in (
                ("log Z", s.logz[i:i + 1], np.array([r.logz]), tz * one),
                ("distill log Z", loss.logz[i:i + 1], np.array([r.logz]), tz * one),
                ("step log Z", step.logz[i:i + 1], np.array([r.logz]), tz * one),
                ("entropy", s.entropy[i:i + 1], np.array([r.entropy]), 2 * tz * one),
                ("log p", s.logp[i], r.logp(ids[i]), 2 * tz * np.ones(K)),
                ("alternatives", s.top_logp[i], top[1], 2 * tz * np.ones(4)),
                ("loss", loss.loss[i:i + 1], np.array([r.distill(ids[i], logits[i].astype(np.float64))]),
                 (2 * tz + 64 * U) * one),
                ("step loss", step.loss[i:i + 1], np.array([r.distill(ids[i], logits[i].astype(np.float64))]),
                 (2 * tz + 64 * U) * one)):
            close(to_np(got), want, tol, what)
        lp = np.where(r.present, r.x - r.logz, 0.0)
        p = np.where(r.present, np.exp(lp), 0.0)
        wt = np.where(r.present, np.abs(h_rows[i].astype(np.complex128)), 1.0)
        with np.errstate(over="ignore", invalid="ignore"):
            rel = np.expm1(4 * tz) + 16 * U
            low = scale * 2.0 ** -126 * (np.abs(g[i]).sum() + abs(h[i]) * 128 + abs(w[i])) if grad_floor else 0.0
            for what, got, (want, mag), he in (
                    ("score gradient", gs[i], r.score_grad(ids[i], g[i], h[i]), abs(h[i])),
                    ("distill gradient", gd[i], r.distill_grad(ids[i], logits[i].astype(np.float64), w[i]), 0.0),
                    ("step gradient", step.grad[i].cpu().numpy(),
                     r.distill_grad(ids[i], logits[i].astype(np.float64), w[i]), 0.0)):
                assert np.isfinite(got).all(), what
                tol = rel * mag + 2 / wt * (scale * he * 2 * tz * p * (1 + rel) + low) + OUT_MIN["c64"]
                tol += OUT_EPS["c64"] * np.abs(want)
                close(got, want, np.where(np.isnan(tol), INF, tol), f"{what} of row {i}")


@pytest.mark.parametrize("R,V", [(9, 64), (9, 1500), (9, 9001), (3, 32768), (2, 400001), (470, 701), (2500, 65)],
                         ids=lambda v: str(v))
@pytest.mark.parametrize("scale", [6.0, 16.0, 20.0, 32.0, 64.0, 1000.0, 5000.0, 2.0 ** 20, 2.0 ** 40])
def test_amplitudes_at_low_temperature(scale, R, V):
    """A quotient of two weights that is small has a power that is not: random
    rows, sorted ones (a new largest weight in every vector), equal ones, and
    ones that differ by their last bits."""
    import torch
    rng = np.random.default_rng(V)
    rows = make_rows(rng, R, V, "c64")
    order = (rows.real.square() + rows.imag.square()).argsort(dim=1)
    rows[1] = rows[1, order[1]]
    rows[2 % R] = rows[2 % R, order[2 % R].flip(0)]
    if R > 3:
        rows[3] = 0.125
    if R > 4:
        rows[4] = 0.25 * (1 + 2.0 ** -23 * torch.from_numpy(rng.integers(0, 4, size=V).astype(np.float32)))
    _check_amplitudes(rows[:9], scale, rng, grad_floor=True)
    if R > 9:       # the kernels that many rows take
        ids = torch.from_numpy(rand_ids(rng, R, 6, V)).cuda()
        d, few = rows.cuda(), rows[:9].cuda()
        one = torch.ones((R, 6), device="cuda")
        ids[:9] = (few.real.square() + few.imag.square()).argmax(dim=1)[:, None]
        many = tn.Outcomes(V, torch.complex64, max_rows=R, top=4, scale=scale)
        less = tn.Outcomes(V, torch.complex64, max_rows=9, top=4, scale=scale)
        a, b = many.score(d, ids), less.score(few, ids[:9])
        assert (a.top_ids[:9] == b.top_ids).all() and torch.isfinite(a.logz).all()
        torch.testing.assert_close(a.logz[:9], b.logz, rtol=4 * U, atol=1e-5)
        torch.testing.assert_close(a.entropy[:9], b.entropy, rtol=1e-4, atol=1e-5)
        a = many.distill_step(d, ids, one, one[:, 0].contiguous())
        b = less.distill_step(few, ids[:9], one[:9], one[:9, 0].contiguous())
        torch.testing.assert_close(a.logz[:9], b.logz, rtol=4 * U, atol=1e-5)
        assert torch.isfinite(a.loss).all() and torch.isfinite(torch.view_as_real(a.grad)).all()


@pytest.mark.parametrize("V", [64, 1500, 40001])
@pytest.mark.parametrize("scale", [0.7, 1.0])
def test_gradients_of_tiny_amplitudes(scale, V):
    """The gradient at an amplitude of 2^-60 is 2^60 and more, and its weight's
    reciprocal times a loss scale of 2^16 beyond fp32."""
    import torch
    rng = np.random.default_rng(V)
    R, K = 4, 5
    a = rng.standard_normal((R, V)) + 1j * rng.standard_normal((R, V))
    a *= 2.0 ** -60 / np.abs(a).max(axis=1, keepdims=True)
    a[np.abs(a) < 2.0 ** -62.9] = 0
    a[1, 0] = 1.0
    rows = torch.from_numpy(a.astype(np.complex64))
    h_rows = to_np(rows)
    ids = np.stack([rng.choice(np.flatnonzero(h_rows[i]), K) for i in range(R)])
    g = (2.0 ** 16 * rng.standard_normal((R, K))).astype(np.float32)
    w = (2.0 ** 16 * rng.standard_normal(R)).astype(np.float32)
    logits = rng.standard_normal((R, K)).astype(np.float32)
    d = rows.cuda()
    d_ids, d_g, d_w, d_l = (torch.from_numpy(x).cuda() for x in (ids, g, w, logits))
    op = tn.Outcomes(V, torch.complex64, max_rows=R, scale=scale)
    s = op.score(d, d_ids)
    got = {"score": op.score_grad(d, d_ids, s.logz, s.entropy, d_g),
           "distill": op.distill_grad(d, d_ids, d_l, s.logz, d_w),
           "step": op.distill_step(d, d_ids, d_l, d_w).grad}
    for i in range(R):
        r = Row(h_rows[i], None, scale)
        loss = r.distill_grad(ids[i], logits[i].astype(np.float64), w[i])
        for what, (want, mag) in (("score", r.score_grad(ids[i], g[i])), ("distill", loss), ("step", loss)):
            tol = (4 * tol_logz(r) + 16 * U) * mag + OUT_EPS["c64"] * np.abs(want) + OUT_MIN["c64"]
            assert np.isfinite(to_np(got[what])[i]).all(), what
            close(to_np(got[what])[i], want, tol, what + " gradient")


@pytest.mark.parametrize("V", [64, 1500, 9001, 400001])
@pytest.mark.parametrize("scale", [0.7, 1.0, 2.5, 6.0, 16.0, 2.0 ** 20])
@pytest.mark.parametrize("largest", [-90, -101, -115, -125])
def test_tiny_amplitudes(largest, scale, V):
    """Rows whose largest weight is 2^largest (a hundred qubits and more), at
    scales whose powers of such weights are below fp32's range; one of them
    ends, one begins with an ordinary weight."""
    import torch
    rng = np.random.default_rng(V)
    a = rng.standard_normal((5, V)) + 1j * rng.standard_normal((5, V))
    a *= 2.0 ** (largest / 2) / np.abs(a).max(axis=1, keepdims=True)
    small = np.abs(a) < 2.0 ** -62.9          # weights are normal numbers, or 0
    a[small] = 0
    a[1, V - 1] = 0.25
    a[2, 0] = 0.25
    _check_amplitudes(torch.from_numpy(a.astype(np.complex64)), scale, rng, grad_floor=True)


@pytest.mark.parametrize("R,V", [(9, 64), (9, 1500), (4, 40001), (1, 400001)], ids=lambda v: str(v))
@pytest.mark.parametrize("scale", [1.0, 2.0, 4.0, 8.0])
def test_gradients_of_unlikely_amplitudes(scale, R, V):
    """Probabilities below 2^-126 whose gradient, p / |a|, is a normal number."""
    import torch
    rng = np.random.default_rng(V)
    a = rng.standard_normal((R, V)) + 1j * rng.standard_normal((R, V))
    a *= 2.0 ** rng.uniform(-35.0, 0.0, size=(R, V))
    _check_amplitudes(torch.from_numpy(a.astype(np.complex64)), scale, rng, grad_floor=False)


@pytest.mark.parametrize("R,V", [(9, 64), (9, 1500), (4, 40001), (1, 400001)], ids=lambda v: str(v))
@pytest.mark.parametrize("lo,hi", [(-62, 0), (-62, 62), (0, 62), (-10, 60)])
@pytest.mark.parametrize("scale", [2.0 ** -40, 0.001, 0.01, 0.05, 0.125, 0.25, 0.3])
def test_amplitudes_at_high_temperature(scale, lo, hi, R, V):
    """Weights up to 2^250 apart, whose powers are not far from each other;
    ascending, descending and random."""
    import torch
    rng = np.random.default_rng(V)
    size = 2.0 ** rng.uniform(lo, hi, size=(R, V))
    size[0] = np.sort(size[0])
    size[-1] = -np.sort(-size[-1])
    a = size * np.exp(2j * np.pi * rng.random((R, V)))
    _check_amplitudes(torch.from_numpy(a.astype(np.complex64)), scale, rng, grad_floor=False)


@pytest.mark.parametrize("R,V", [(600, 1000), (3, 3001), (2, 60000), (400, 40001), (1, 900001)],
                         ids=lambda v: str(v))
def test_step_keeps_small_bf16_gradients(R, V):
    """bf16 reaches below the least probability of one exponential: logits 80
    to 100 below the largest have a gradient with a loss scale of 2^20, whichever
    way the step takes, the same as from the two calls."""
    import torch
    z = np.full((R, V), 100.0)
    z[:, 1:] -= np.linspace(80, 100, V - 1)
    rows = torch.from_numpy(z.astype(np.float32)).bfloat16()
    ids = np.zeros((R, 1), np.int64)
    w = np.full(R, 2.0 ** 20, np.float32)
    d, d_ids, d_l = rows.cuda(), torch.from_numpy(ids).cuda(), torch.zeros((R, 1), device="cuda")
    op = tn.Outcomes(V, torch.bfloat16, max_rows=R)
    s = op.distill(d, d_ids, d_l)
    step = to_np(op.distill_step(d, d_ids, d_l, torch.from_numpy(w).cuda()).grad)
    both = to_np(op.distill_grad(d, d_ids, d_l, s.logz, torch.from_numpy(w).cuda()))
    r = Row(to_np(rows)[0], None, 1.0)
    want, mag = r.distill_grad(ids[0], np.zeros(1), w[0])
    tol = (4 * tol_logz(r) + 16 * U) * mag + OUT_EPS["bf16"] * np.abs(want) + OUT_MIN["bf16"]
    assert (np.abs(want[1:]) > 1e-38).sum() > V // 2
    for what, got in (("step", step), ("distill", both)):
        close(got, np.broadcast_to(want, (R, V)), np.broadcast_to(tol, (R, V)), what + " gradient")


@pytest.mark.parametrize("V", [100, 30000, 900001])
@pytest.mark.parametrize("scale", [1.0, 1.25, 100.0])
def test_large_teacher_logits(scale, V):
    """A teacher whose logits leave fp32 when scaled: the lowest value alone
    (uniform), beside ordinary ones (probability 0), and large positive ones
    (the largest is certain)."""
    rng = np.random.default_rng(V)
    low = np.finfo(np.float32).min
    ids = np.stack([rng.permutation(V)[:4] for _ in range(5)]).astype(np.int64)
    t = np.array([[low] * 4, [low, 0.5, low, 0.25], [3e38, 2e38, 3e38, -3e38], [low, -INF, low, -INF],
                  [1e38, 0.0, -1e38, 1e38]], np.float32)
    run_all(make_rows(rng, 5, V, "f32"), "f32", None, 0, (ids, t), teacher_scale=scale, rng=rng)


@pytest.mark.parametrize("t,scale,offset", [
    ("f32", 1.0, 0.0), ("f32", 1.0, 1e4), ("f32", 0.7, 1e7), ("f32", 1.25, -1e9), ("f32", 1.0, -3.4e38),
    ("f32", 1.25, -3.4e38), ("f32", 1.25, 3.4e38), ("bf16", 1.0, -1e9), ("bf16", 1.25, -3.38e38),
    ("f16", 1.0, -65504.0), ("f16", 2.0, -65504.0), ("c64", 2.0 ** 20, 0.0), ("c64", 2.0 ** 40, 0.0)])
@pytest.mark.parametrize("R,V", [(5, 60), (4, 4001), (3, 50001), (1, 1500001), (2500, 33)], ids=lambda v: str(v))
def test_log_probabilities_beside_large_logits(R, V, t, scale, offset):
    """log p and the loss are differences, whatever log Z rounds to: of logits far
    from 0, of rows that one value fills (also where scale z leaves fp32), of
    equal amplitudes at large scales.

    Bounds, without M: two roundings of scale (z - z0), the exponential's error
    for every term of the sum, weighted by p (1 + H), and ln s: 16 u (1 + |log p|
    + H).  The reference is of the logits less their largest, in 64 bits."""
    import torch
    rng = np.random.default_rng(V)
    if t == "c64":
        rows = torch.full((R, V), 0.3 + 0.1j, dtype=torch.complex64)
    else:
        z = 3.0 * rng.standard_normal((R, V)) if abs(offset) < 1e38 else np.zeros((R, V))
        rows = torch.from_numpy((z + offset).astype(np.float32)).to(torch_type(t))
        rows[0] = offset
    h = np.zeros((min(R, 5), V)) if t == "c64" else to_np(rows)[:5].astype(np.float64)
    ids, logits = rand_ids(rng, R, 4, V), rng.standard_normal((R, 4)).astype(np.float32)
    d, d_ids, d_l = rows.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(logits).cuda()
    op = tn.Outcomes(V, torch_type(t), max_rows=R, top=3, scale=scale)
    s = op.score(d, d_ids)
    loss = op.distill(d, d_ids, d_l).loss
    step = op.distill_step(d, d_ids, d_l, torch.ones(R, device="cuda")).loss
    for i in range(len(h)):
        r = Row(h[i] - h[i].max(), None, scale)
        unit = 16 * U * (1 + r.entropy)
        lp = r.logp(ids[i])
        close(to_np(s.logp)[i], lp, unit + 16 * U * np.abs(lp), "log p")
        top = r.top(3)
        assert (to_np(s.top_ids)[i] == top[0]).all()
        close(to_np(s.top_logp)[i], top[1], unit + 16 * U * np.abs(top[1]), "alternatives")
        want = np.array([r.distill(ids[i], logits[i].astype(np.float64))])
        far = np.abs(np.where(ids[i] < 0, 0.0, lp)).max()
        for what, got in (("loss", loss), ("step loss", step)):
            close(to_np(got)[i:i + 1], want, np.array([2 * unit + 32 * U * (far + 8.0)]), what)


@pytest.mark.parametrize("layout", ["aligned", "misaligned", "strided"])
@pytest.mark.parametrize("t,scale,value", [("f32", 1.0, -1e9), ("f32", 1.25, -3.4e38), ("f32", 0.7, 1e30),
                                           ("bf16", 1.0, -1e9), ("bf16", 1.25, -3.38e38), ("f16", 1.0, -65504.0),
                                           ("c64", 2.0 ** 20, 0.3), ("c64", 2.0 ** 40, 0.3)])
@pytest.mark.parametrize("R,V", [(3, 60), (2, 4001), (2, 50001), (500, 700)], ids=lambda v: str(v))
def test_step_of_filled_rows(R, V, t, scale, value, layout):
    """Rows that one large value fills are uniform, for the entries that the
    teacher names and those at the rows' ends as for all others.

    Bounds: p = 1 / V to the rounding of ln V (8 u (1 + ln V)), the gradient's
    type, and the factors' roundings."""
    import torch
    rng = np.random.default_rng(V)
    buf = torch.zeros((R, 2 * V + 18), dtype=torch_type(t), device="cuda")
    d = {"aligned": torch.zeros((R, V), dtype=torch_type(t), device="cuda"), "misaligned": buf[:, 1:V + 1],
         "strided": buf[:, ::2][:, :V]}[layout]
    d.fill_(value)
    ids, logits = rand_ids(rng, R, 5, V), rng.standard_normal((R, 5)).astype(np.float32)
    ids[0, :2] = [0, V - 1]
    w = rng.standard_normal(R).astype(np.float32)
    op = tn.Outcomes(V, torch_type(t), max_rows=R, scale=scale)
    got = op.distill_step(d, torch.from_numpy(ids).cuda(), torch.from_numpy(logits).cuda(),
                          torch.from_numpy(w).cuda())
    grad = to_np(got.grad)
    if t == "c64":      # 2 a / |a|^2 dL/dz, of a real amplitude
        assert (grad.imag == 0).all()
        grad = grad.real.astype(np.float64) * float(np.float32(value)) / 2.0
    eps = 16 * U * (1 + np.log(V)) + OUT_EPS[t]
    for i in range(min(R, 4)):
        want, mag = Row(np.zeros(V, np.float32), None, scale).distill_grad(ids[i], logits[i].astype(np.float64), w[i])
        close(grad[i].astype(np.float64), want, eps * mag + OUT_MIN[t], f"gradient of row {i}")
    np.testing.assert_allclose(to_np(got.loss)[0], Row(np.zeros(V, np.float32), None, 1.0).distill(
        ids[0], logits[0].astype(np.float64)), rtol=1e-5, atol=1e-5)


def test_absent_teacher_outcomes():
    """A teacher's outcome with an unmasked -inf logit: infinite loss; the
    same outcome masked: left out of the teacher."""
    import torch
    rng = np.random.default_rng(2)
    rows = make_rows(rng, 3, 100, "f32")
    rows[:, 10] = -INF
    ids = np.array([[10, 20], [20, 30], [10, -1]], np.int64)
    t = np.zeros((3, 2), np.float32)
    run_all(rows, "f32", None, 0, (ids, t))
    keep = torch.ones((3, 100), dtype=torch.bool)
    keep[:, 10] = False
    run_all(rows, "f32", None, 0, (ids, t), mask=keep)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("V", [40, 30011])
def test_repeated_ids_add_up(V, t):
    rng = np.random.default_rng(21)
    R = 4
    ids = rng.integers(0, 6, size=(R, 256)).astype(np.int64)
    given = rng.integers(0, 5, size=(R, 256)).astype(np.int64)
    run_all(make_rows(rng, R, V, t), t, given, 0,
            (ids, rng.standard_normal((R, 256)).astype(np.float32)), rng=rng)


@pytest.mark.parametrize("V", [60, 70001])
def test_given_shapes_and_none(V):
    """[R] ids, all -1, and no given at all."""
    rng = np.random.default_rng(4)
    rows = make_rows(rng, 3, V, "bf16")
    run_all(rows, "bf16", rng.integers(0, V, size=3).astype(np.int64), 0, None, rng=rng)
    run_all(rows, "bf16", np.full((3, 2), -1, np.int64), 1, None, rng=rng)
    run_all(rows, "bf16", None, 2, (np.full((3, 2), -1, np.int64), np.zeros((3, 2), np.float32)), rng=rng)


@pytest.mark.parametrize("V", [50, 30000])
def test_ids_out_of_range_are_reported(V):
    """Ids outside [-1, cols) read nothing: NaN in their places and a device
    status, which the next check finds cleared."""
    import torch
    rng = np.random.default_rng(6)
    rows = make_rows(rng, 3, V, "f32").cuda()
    op = tn.Outcomes(V, torch.float32, max_rows=3)
    given = torch.tensor([[0, V], [1, -1], [-2, 3]]).cuda()
    s = op.score(rows, given)
    torch.cuda.synchronize()
    with pytest.raises(tn.TNError) as e:
        op.check()
    assert e.value.status == tn.TN_EDEVICE
    op.check()
    lp = to_np(s.logp)
    assert np.isnan(lp[0, 1]) and np.isnan(lp[2, 0]) and np.isfinite(lp[[0, 1, 1, 2], [0, 0, 1, 1]]).all()
    g = op.score_grad(rows, given, s.logz, s.entropy, torch.ones_like(s.logp))
    with pytest.raises(tn.TNError):
        op.check()
    assert np.isfinite(to_np(g)).all()
    r = op.distill(rows, given, torch.zeros_like(s.logp))
    with pytest.raises(tn.TNError):
        op.check()
    loss = to_np(r.loss)
    assert np.isnan(loss[[0, 2]]).all() and np.isfinite(loss[1])


@pytest.mark.parametrize("z", [1e10, -1e10, -1e30])
@pytest.mark.parametrize("scale", [0.7, 1.0, 1.25])
@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("V", [75, 4001, 50001])
def test_gradients_of_large_logits(V, t, scale, z):
    """log p = scale z - log Z with the product rounded, in every entry: where
    log Z is the rounded product itself, p is 1 and not e to the power of that
    rounding (512 at 1e10).  Rows without weight have no gradient."""
    import torch
    R = 2
    rng = np.random.default_rng(V)
    rows = torch.full((R, V), z).to(torch_type(t)).cuda()
    c = np.float32(scale)
    logz = rows[:, 0].float() * float(c)
    given = torch.from_numpy(rand_ids(rng, R, 2, V)).cuda()
    given[0, 0] = 3
    g = torch.tensor([[0.75, 0.5], [0.0, 0.0]], device="cuda")
    h = torch.tensor([0.5, 0.0], device="cuda")
    op = tn.Outcomes(V, torch_type(t), max_rows=R, scale=scale)
    zero = torch.zeros(R, device="cuda")
    total = (g * (given >= 0)).sum(dim=1, keepdim=True)
    at = torch.zeros((R, V), device="cuda").scatter_add_(1, given.clamp(min=0), g * (given >= 0))
    for he in (None, h):        # with log p = 0 and an entropy given as 0 it adds nothing
        got = op.score_grad(rows, given, logz, zero, g, he).float()
        close(to_np(got), to_np(float(c) * (at - total)), np.full((R, V), 8 * U + OUT_EPS[t]), "score gradient")
    w = torch.tensor([0.25, 0.0], device="cuda")
    ids = given[:, :1].contiguous()
    ids[ids < 0] = 0
    got = op.distill_grad(rows, ids, torch.zeros((R, 1), device="cuda"), logz, w).float()
    want = torch.full((R, V), float(c), device="cuda").scatter_add_(1, ids, torch.full((R, 1), -float(c), device="cuda"))
    close(to_np(got), to_np(want * w[:, None]), np.full((R, V), 8 * U + OUT_EPS[t]), "distill gradient")


@pytest.mark.parametrize("t", ["f32", "c64"])
def test_gradients_against_differences(t):
    """Central differences of the 64-bit scores and loss along single
    entries, at steps whose truncation (h^2) and cancellation (2^-53 / h) are
    both below 1e-8."""
    import torch
    rng = np.random.default_rng(8)
    V, c = 23, 0.8
    rows = make_rows(rng, 1, V, t)
    h_row = to_np(rows)[0]
    given = np.array([[3, 3, 11]], np.int64)
    g, he = np.array([0.3, -1.1, 0.7]), 0.4
    ids, tl = np.array([[2, 5, 5, 19]], np.int64), np.array([[0.5, -1.0, 0.1, 2.0]], np.float32)

    def score(row):
        r = Row64(row, c)
        return float(g @ r.logp(given[0]) + he * r.entropy)

    def loss(row):
        return Row64(row, c).distill(ids[0], tl[0].astype(np.float64))

    op = tn.Outcomes(V, torch_type(t), scale=c)
    d = rows.cuda()
    s = op.score(d, torch.from_numpy(given).cuda())
    gs = to_np(op.score_grad(d, torch.from_numpy(given).cuda(), s.logz, s.entropy,
                             torch.from_numpy(g[None].astype(np.float32)).cuda(),
                             torch.tensor([he], dtype=torch.float32).cuda()))[0]
    gd = to_np(op.distill_step(d, torch.from_numpy(ids).cuda(), torch.from_numpy(tl).cuda(),
                               torch.ones(1).cuda()).grad)[0]
    base = h_row.astype(np.complex128 if t == "c64" else np.float64)
    eps = 1e-4 * (np.abs(base).mean() if t == "c64" else 1.0)
    for got, fn in ((gs, score), (gd, loss)):
        scale = np.abs(got).max()
        for v in range(V):
            for unit, part in ((1.0, np.real), (1j, np.imag)) if t == "c64" else ((1.0, np.real),):
                up, dn = base.copy(), base.copy()
                up[v] += eps * unit
                dn[v] -= eps * unit
                want = (fn(up) - fn(dn)) / (2 * eps)
                assert abs(part(got[v]) - want) <= 2e-5 * scale, (v, unit)


class Row64(Row):
    """The definition without the 32-bit order value, for differences."""

    def __init__(self, row, scale):
        super().__init__(row, None, scale)
        if np.iscomplexobj(row):
            self.x = scale * np.log(row.real ** 2 + row.imag ** 2)
            m = self.x.max()
            self.logz = m + np.log(np.exp(self.x - m).sum())
            lp = self.x - self.logz
            self.entropy = -(np.exp(lp) * lp).sum()


@pytest.mark.parametrize("shape", [(3, 1000), (2, 200001)], ids=lambda s: f"{s[0]}x{s[1]}")
def test_results_do_not_vary(shape):
    """Bitwise equal from run to run, and on a handle made for more rows."""
    import torch
    R, V = shape
    rng = np.random.default_rng(12)
    rows = make_rows(rng, R, V, "bf16").cuda()
    given = torch.from_numpy(rand_ids(rng, R, 3, V)).cuda()
    ids, t = rand_teacher(rng, R, 12, V)
    ids, t, w = torch.from_numpy(ids).cuda(), torch.from_numpy(t).cuda(), torch.ones(R).cuda()
    runs = []
    for max_rows in (R, R, 50):
        op = tn.Outcomes(V, torch.bfloat16, max_rows=max_rows, top=9)
        for _ in range(3):
            s = op.score(rows, given)
            d = op.distill_step(rows, ids, t, w)
            runs.append([to_np(x) for x in (*s, *d)])
    for r in runs[1:]:
        for a, b in zip(runs[0], r):
            assert a.tobytes() == b.tobytes()


def test_own_stream_and_graph():
    """On a side stream, and captured into a CUDA graph and replayed on new
    contents."""
    import torch
    rng = np.random.default_rng(13)
    V, R = 100003, 2
    a, b = make_rows(rng, R, V, "f32").cuda(), make_rows(rng, R, V, "f32").cuda()
    op = tn.Outcomes(V, torch.float32, max_rows=R, top=4)
    want = [to_np(x) for r in (a, b) for x in op.score(r)[:2] + op.score(r)[3:]]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s = op.score(a, stream=side)
    side.synchronize()
    for x, y in zip((s.logz, s.entropy, s.top_ids, s.top_logp), want[:4]):
        assert (to_np(x) == y).all()
    buf, out = a.clone(), op.score(a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.score(buf, out=out)
    for rows, w in ((b, want[4:]), (a, want[:4])):
        buf.copy_(rows)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip((out.logz, out.entropy, out.top_ids, out.top_logp), w):
            assert (to_np(x) == y).all()


CALLS = ["score", "score_grad", "distill", "distill_grad", "distill_step"]


def _call(op, name, x, stream=None):
    """One call on the inputs x, its outputs as a list."""
    kw = {"mask": x["mask"], "stream": stream}
    if name == "score":
        r = op.score(x["rows"], x["ids"], **kw)
    elif name == "score_grad":
        r = (op.score_grad(x["rows"], x["ids"], x["logz"], x["entropy"], x["logits"], x["w"], **kw),)
    elif name == "distill":
        r = op.distill(x["rows"], x["ids"], x["logits"], **kw)[:2]
    elif name == "distill_grad":
        r = (op.distill_grad(x["rows"], x["ids"], x["logits"], x["logz"], x["w"], **kw),)
    else:
        r = op.distill_step(x["rows"], x["ids"], x["logits"], x["w"], **kw)
    return list(r)


def _inputs_of_calls(t, R, V, seed):
    import torch
    rng = np.random.default_rng(seed)
    x = {"rows": make_rows(rng, R, V, t), "mask": torch.from_numpy(rng.random((R, V)) < 0.8),
         "ids": torch.from_numpy(rand_ids(rng, R, 5, V)),
         "logits": torch.from_numpy(rng.standard_normal((R, 5)).astype(np.float32)),
         "w": torch.from_numpy(rng.standard_normal(R).astype(np.float32))}
    x = {k: v.cuda() for k, v in x.items()}
    op = tn.Outcomes(V, torch_type(t), max_rows=R, top=4, scale=0.7)
    s = op.score(x["rows"], mask=x["mask"])
    x["logz"], x["entropy"] = s.logz, s.entropy
    return x


@pytest.mark.parametrize("t,R,V", [("bf16", 5, 300), ("f32", 3, 20011), ("c64", 2, 400001), ("bf16", 700, 9001)])
@pytest.mark.parametrize("name", CALLS)
def test_every_call_in_a_graph(name, t, R, V):
    """Captured on a fresh handle (its first call but for the workspace) and
    replayed on new contents, bit by bit as the call itself."""
    import torch
    xs = [_inputs_of_calls(t, R, V, seed) for seed in (1, 2)]
    plain = tn.Outcomes(V, torch_type(t), max_rows=R, top=4, scale=0.7)
    want = [[to_np(o) for o in _call(plain, name, x)] for x in xs]
    op = tn.Outcomes(V, torch_type(t), max_rows=R, top=4, scale=0.7)
    op.bind_workspace()
    buf = {k: v.clone() for k, v in xs[0].items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _call(op, name, buf)
    for x, w in ((xs[1], want[1]), (xs[0], want[0]), (xs[1], want[1])):
        for k, v in x.items():
            buf[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, w):
            assert to_np(a).tobytes() == b.tobytes()


@pytest.mark.parametrize("t,R,V", [("bf16", 5, 300), ("f32", 64, 200003), ("c64", 700, 9001)])
@pytest.mark.parametrize("name", CALLS)
def test_every_call_on_a_side_stream(name, t, R, V):
    """Given as a torch stream, as its handle, and as the current stream; inputs
    are dropped while it still works, and what is allocated next is filled."""
    import torch
    base = _inputs_of_calls(t, R, V, 3)
    plain = tn.Outcomes(V, torch_type(t), max_rows=R, top=4, scale=0.7)
    want = [to_np(o) for o in _call(plain, name, base)]
    side = torch.cuda.Stream()
    for how in ("stream", "handle", "current"):
        op = tn.Outcomes(V, torch_type(t), max_rows=R, top=4, scale=0.7)
        op.bind_workspace()
        for _ in range(4):
            x = {k: v.clone() for k, v in base.items()}
            side.wait_stream(torch.cuda.current_stream())
            if how == "current":
                with torch.cuda.stream(side):
                    got = _call(op, name, x)
                for v in x.values():
                    v.record_stream(side)
            else:
                got = _call(op, name, x, stream=side if how == "stream" else side.cuda_stream)
            sizes = [(v.shape, v.dtype) for v in x.values()]
            del x
            junk = [torch.ones(s, dtype=d, device="cuda") for s, d in sizes]
            side.synchronize()
            for a, b in zip(got, want):
                assert to_np(a).tobytes() == b.tobytes()
            torch.cuda.synchronize()
            del junk, got


def test_no_rows():
    import torch
    op = tn.Outcomes(100, torch.float32, max_rows=4, top=3)
    s = op.score(torch.empty((0, 100), device="cuda"))
    assert s.logz.shape == (0,) and s.top_ids.shape == (0, 3)
    e = torch.empty((0, 2), dtype=torch.int64, device="cuda")
    d = op.distill_step(torch.empty((0, 100), device="cuda"), e, torch.empty((0, 2), device="cuda"),
                        torch.empty(0, device="cuda"))
    assert d.grad.shape == (0, 100)


def test_offsets_past_32_bits():
    """Rows whose last entries lie past 2^32 bytes and 2^31 entries."""
    import torch
    V, R = 3000001, 720                     # 2.16e9 entries of bf16: 4.3 GB
    rows = torch.zeros((R, V), dtype=torch.bfloat16, device="cuda")
    rows[R - 1, V - 2] = 9.0
    rows[R - 1, V - 1] = 8.0
    rows[0, 5] = 7.0
    op = tn.Outcomes(V, torch.bfloat16, max_rows=R, top=2)
    given = torch.full((R, 1), V - 2, dtype=torch.int64, device="cuda")
    s = op.score(rows, given)
    assert to_np(s.top_ids[R - 1]).tolist() == [V - 2, V - 1]
    assert to_np(s.top_ids[0]).tolist() == [5, 0]
    lz = np.log(V - 2 + np.exp(9.0) + np.exp(8.0))
    np.testing.assert_allclose(float(s.logz[R - 1]), lz, rtol=1e-6)
    np.testing.assert_allclose(float(s.logp[R - 1, 0]), 9.0 - lz, rtol=1e-5)
    g = op.score_grad(rows, given, s.logz, s.entropy, torch.ones((R, 1), device="cuda"))
    np.testing.assert_allclose(float(g[R - 1, V - 2]), 1 - np.exp(9.0 - lz), rtol=2.0 ** -8)
    np.testing.assert_allclose(float(g[R - 1, V - 1]), -np.exp(8.0 - lz), rtol=2.0 ** -8)
    np.testing.assert_allclose(float(g[R - 1, 0]), -np.exp(-lz), rtol=2.0 ** -8)


def test_refusals():
    import torch
    op = tn.Outcomes(64, torch.float32, max_rows=2, top=3)
    ok = torch.zeros((2, 64), device="cuda")
    ids, t, w = torch.zeros((2, 4), dtype=torch.int64).cuda(), torch.zeros((2, 4)).cuda(), torch.ones(2).cuda()
    bad_calls = [
        lambda: op.score(ok.double()),
        lambda: op.score(ok.cpu()),
        lambda: op.score(ok[:, :63]),
        lambda: op.score(ok[None]),
        lambda: op.score(ok, ids.int()),
        lambda: op.score(ok, ids.cpu()),
        lambda: op.score(ok, ids[:1]),
        lambda: op.score(ok, ids.t().contiguous().t()),
        lambda: op.score(ok, mask=ok),
        lambda: op.score(ok, mask=torch.ones((2, 64), dtype=torch.bool)),
        lambda: op.score_grad(ok, ids, w, w, t[:, :2].contiguous()),
        lambda: op.score_grad(ok, ids, w.double(), w, t),
        lambda: op.score_grad(ok, ids, w, w, t, w[:1]),
        lambda: op.score_grad(ok, ids, w, w, t, out=ok[:1]),
        lambda: op.distill(ok, ids, t.double()),
        lambda: op.distill(ok, ids, t[:, :3].contiguous()),
        lambda: op.distill_step(ok, ids, t, w.cpu()),
        lambda: tn.Outcomes(64, torch.complex64, max_rows=2).score(torch.zeros((2, 64), dtype=torch.complex64).cuda().conj()),
        lambda: tn.Outcomes(64, torch.float64),
    ]
    for f in bad_calls:
        with pytest.raises((ValueError, RuntimeError)):
            f()
    # refused by the library
    for f in (lambda: op.score(torch.zeros((3, 64), device="cuda")),            # more rows than made for
              lambda: op.score(ok, torch.zeros((2, 257), dtype=torch.int64).cuda()),
              lambda: op.distill(ok, ids, t, teacher_scale=0.0),
              lambda: op.distill(ok, ids, t, teacher_scale=INF),
              lambda: op.score(torch.zeros((2, 1), device="cuda").expand(2, 64))):
        with pytest.raises(tn.TNError) as e:
            f()
        assert e.value.status == tn.TN_EINVAL
    with pytest.raises(tn.TNError) as e:
        tn.tn_outcomes_score(tn.Outcomes(64, torch.float32).handle,
                             tn.tn_rows(ok.data_ptr(), 1, 64, 1, None, 0, 0), None, 0, None,
                             w.data_ptr(), w.data_ptr(), 0, None, None)
    assert e.value.status == tn.TN_ENOMEM
    torch.cuda.synchronize()
    op.check()


def test_handle_may_go_before_its_work():
    """A handle and its inputs dropped while a side stream still works with
    them; what is allocated next does not land in their memory."""
    import torch
    rng = np.random.default_rng(17)
    rows = make_rows(rng, 64, 200003, "f32").cuda()
    want = tn.Outcomes(200003, torch.float32, max_rows=64, top=20).score(rows)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        op = tn.Outcomes(200003, torch.float32, max_rows=64, top=20)
        op.score(rows)
        nbytes = op.workspace_bytes
        side.wait_stream(torch.cuda.current_stream())
        got = [op.score(rows, stream=side) for _ in range(5)]
        del op
        junk = [torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
        side.synchronize()
        torch.cuda.synchronize()
        del junk
        for s in got:
            for x, y in zip(s[:2] + s[3:], want[:2] + want[3:]):
                assert (x == y).all()
