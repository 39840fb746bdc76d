"""The definitions of the outcome operators in 64 bits, row by row in numpy.
Shares no code with the library."""
import numpy as np

INF = float("inf")


def row_logits(row):
    """(order value, logit) of a row: complex64 amplitudes, or real logits."""
    if np.iscomplexobj(row):
        re, im = row.real.astype(np.float32), row.imag.astype(np.float32)
        with np.errstate(over="ignore", under="ignore", invalid="ignore", divide="ignore"):
            w = (re * re + im * im)          # the order is defined in 32 bits
            a = row.astype(np.complex128)
            z = np.log(a.real ** 2 + a.imag ** 2)
        return w.astype(np.float64), np.where(w == 0, -INF, z)
    z = row.astype(np.float64) + 0.0
    return z, z


class Row:
    def __init__(self, row, keep, scale):
        self.row, self.scale = row, scale
        self.order, z = row_logits(row)
        self.keep = np.ones(row.shape, bool) if keep is None else keep.astype(bool)
        self.present = self.keep & (z != -INF)
        self.x = np.where(self.present, scale * np.where(self.present, z, 0.0), -INF)
        xs = self.x[self.present]
        self.bad = bool(np.isnan(xs).any() or (xs == INF).any())
        self.empty = xs.size == 0
        if self.bad:
            self.logz, self.entropy = np.nan, np.nan
        elif self.empty:
            self.logz, self.entropy = -INF, 0.0
        else:
            m = xs.max()
            self.logz = m + np.log(np.exp(xs - m).sum())
            lp = xs - self.logz
            self.entropy = -(np.exp(lp) * lp).sum()
        # bound of |scale z| for tolerances
        fin = np.abs(xs[np.isfinite(xs)])
        self.mag = float(fin.max()) if fin.size else 0.0

    def logp(self, ids):
        out = np.empty(len(ids))
        for j, i in enumerate(ids):
            if i == -1:
                out[j] = 0.0
            elif i < 0 or i >= len(self.row):
                out[j] = np.nan
            elif not self.present[i]:
                out[j] = -INF
            else:
                out[j] = self.x[i] - self.logz
        return out

    def top(self, k):
        ids, lp = np.full(k, -1, np.int64), np.full(k, -INF)
        if self.bad:
            return ids, np.full(k, np.nan)
        at = np.flatnonzero(self.present)
        best = at[np.argsort(-self.order[at], kind="stable")][:k]
        ids[:len(best)] = best
        lp[:len(best)] = self.x[best] - self.logz
        return ids, lp

    def _finish(self, gz, mag):
        """Gradient of the logits and its error scale, as the row's."""
        gz = np.where(self.present, gz, 0.0)
        mag = np.where(self.present, mag, 0.0)
        if np.iscomplexobj(self.row):
            a = np.where(self.present, self.row, 0.0).astype(np.complex128)
            w = np.where(self.present, a.real ** 2 + a.imag ** 2, 1.0)
            return 2.0 * a / w * gz, 2.0 / np.sqrt(w) * mag
        return gz, mag

    def score_grad(self, ids, g, h=0.0):
        n = len(self.row)
        add, tot = np.zeros(n), 0.0
        absadd, abstot = np.zeros(n), 0.0
        for i, gi in zip(ids, g):
            if 0 <= i < n and self.present[i]:
                add[i] += gi
                absadd[i] += abs(gi)
                tot += gi
                abstot += abs(gi)
        if self.empty:
            return self._finish(np.zeros(n), np.zeros(n))
        lp = np.where(self.present, self.x - self.logz, 0.0)
        p = np.where(self.present, np.exp(lp), 0.0)
        gz = self.scale * (add - p * (tot + h * (lp + self.entropy)))
        mag = self.scale * (absadd + p * (abstot + abs(h) * (np.abs(lp) + self.entropy)))
        return self._finish(gz, mag)

    def teacher(self, ids, t):
        used = [(i, tj) for i, tj in zip(ids, t)
                if 0 <= i < len(self.row) and self.keep[i] and tj != -INF]
        if not used:
            return [], np.zeros(0)
        x = np.array([tj for _, tj in used], dtype=np.float64)
        e = np.exp(x - x.max())
        return [i for i, _ in used], e / e.sum()

    def distill(self, ids, t):
        at, q = self.teacher(ids, t)
        if any(i < -1 or i >= len(self.row) for i in ids):
            return np.nan
        if self.empty or not at:
            return 0.0
        loss = 0.0
        for i, qi in zip(at, q):
            if qi != 0:
                lp = self.x[i] - self.logz if self.present[i] else -INF
                loss += qi * (np.log(qi) - lp)
        return loss

    def distill_grad(self, ids, t, g):
        n = len(self.row)
        at, q = self.teacher(ids, t)
        if self.empty or not at:
            return self._finish(np.zeros(n), np.zeros(n))
        p = np.where(self.present, np.exp(np.where(self.present, self.x - self.logz, 0.0)), 0.0)
        d = np.zeros(n)
        for i, qi in zip(at, q):
            d[i] += qi
        return self._finish(g * self.scale * (p - d), abs(g) * self.scale * (p + d))
