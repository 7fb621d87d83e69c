"""The gated linear recurrence and its gradients, one step after another in 64 bits, with a bound on
what the same computation in 32 bits can be off.

The bound follows the kernels' arithmetic with u = 2^-23 (one step of fp32 relative to the value;
a rounding is half of it):
  v = root^2 / (2 (1 + E)): E = e^-r from a rounded argument, (|r| + 2) u; the sum 0.5 u; its reciprocal root
  1.1 u and root = sqrt(2 c softplus(lam)) 2.5 u, a product 0.5 u, all three doubled by the square, 0.5 u; in all
  (|r| + 11) u of v, and so v times that of a = e^-v, whose exponential or polynomial costs 2 u more:
      e_a = (3 + v (|r| + 11)) u   relative;
  b = m iota x: m is a polynomial in v times sqrt(v), or the root of 1 - a^2, which is off by 24 u at the border
  between the two (half of it in m); iota = 1 / (1 + e^-i) 4 u + |i| u:   e_b = (22 + |r| + |i|) u   relative;
  the state's error E_t = a_t (E_{t-1} + (e_a + u) H_{t-1}) + (e_b + u) |b_t|  with H the recurrence of |b|.
Composing stretches in another order has as many roundings on every path again: E doubled.
y of bf16 is gated by z (1 + tanh(z / 2)) / 2 with tanh.approx, at most 2^-10.98 off relative to tanh and so at most
2^-11.9 |z| off in silu(z); the other gates are as above.
bf16 results are rounded once more, by at most 2^-8 of their value; inputs of bf16 enter as they are.
"""
import numpy as np

U = 2.0 ** -23


def sigmoid(v):
    return np.where(v >= 0, 1 / (1 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1 + np.exp(-np.abs(v))))


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def reference(x, r, i, lam, r_bias=None, i_bias=None, z=None, initial_state=None, lengths=None, reset=None, c=8.0, dy=None,
              dlast=None, bf16=False):
    """Returns {name: (value, bound)}; with dy the gradients too."""
    x, r, i, z, dy = (f64(t) for t in (x, r, i, z, dy))
    lam, r_bias, i_bias, h0, dlast = (f64(t) for t in (lam, r_bias, i_bias, initial_state, dlast))
    B, D, L = x.shape
    n = np.full(B, L) if lengths is None else np.clip(lengths.cpu().numpy().astype(np.int64), 0, L)
    cut = np.zeros((B, L), bool) if reset is None else reset.cpu().numpy() != 0
    r = r + (0 if r_bias is None else r_bias[:, None])
    i = i + (0 if i_bias is None else i_bias[:, None])
    soft = np.logaddexp(0, lam)
    with np.errstate(all="ignore"):
        rho, iota = sigmoid(r), sigmoid(i)
        v = c * soft[:, None] * rho
        a, m = np.exp(-v), np.sqrt(-np.expm1(-2 * v))
        a, m = np.where(cut[:, None], 0, a), np.where(cut[:, None], 1, m)
        ea = (3 + v * (np.abs(r) + 11)) * U
        eb = (22 + np.abs(r) + np.abs(i)) * U
        b = m * iota * x
        h = np.zeros((B, D)) if h0 is None else h0.copy()
        H, E = np.abs(h), np.abs(h) * U
        hs, Es, before, Ebefore = (np.zeros((B, D, L)) for _ in range(4))
        for t in range(L):
            on = (t < n)[:, None]
            before[..., t], Ebefore[..., t] = h, E
            keep = cut[:, t][:, None]  # nothing reaches over a reset, not even a NaN
            new = np.where(keep, 0, a[..., t] * h) + b[..., t]
            E = np.where(on, np.where(keep, 0, a[..., t] * (E + (ea[..., t] + U) * H)) + (eb[..., t] + U) * np.abs(b[..., t]), E)
            H = np.where(on, np.where(keep, 0, a[..., t] * H) + np.abs(b[..., t]), H)
            h = np.where(on, new, h)
            hs[..., t], Es[..., t] = h, E
        inside = (np.arange(L) < n[:, None])[:, None, :]
        half = 2.0 ** -8 if bf16 else 0.5 * U

        def rounded(val, err):
            val, err = np.where(inside, val, 0), np.where(inside, err, 0)
            return val, 2 * err + half * (np.abs(val) + 2 * err) + 1e-30

        gate = 1 if z is None else z * sigmoid(z)
        tanh = 2.0 ** -11.9 * np.abs(z) if bf16 and z is not None else 0
        egate = 0 if z is None else (8 + np.abs(z)) * U
        out = {"y": rounded(hs * gate, (Es + egate * np.abs(hs)) * np.abs(gate) + tanh * np.abs(hs)), "last": (h, 2 * E + 1e-30)}
        if dy is None:
            return out
        if z is not None:
            sig = sigmoid(z)
            slope = sig * (1 + z * (1 - sig))
            out["dz"] = rounded(dy * hs * slope, np.abs(dy) * (Es * np.abs(slope) + np.abs(hs) * (12 + np.abs(z)) * U * sig * (1 + np.abs(z))))
        dv = np.where(inside, dy * gate, 0)
        s = np.zeros((B, D)) if dlast is None else dlast.copy()
        Sa, Sg = np.abs(s), np.abs(s) * U
        dx, dr, di, T, edx, edr, edi, eT = (np.zeros((B, D, L)) for _ in range(8))
        for t in range(L - 1, -1, -1):
            on = (t < n)[:, None]
            keep = cut[:, t][:, None]
            g, eg = dv[..., t] + s, Sg + (egate if z is None else egate[..., t]) * np.abs(dv[..., t]) + U * (np.abs(dv[..., t]) + Sa)
            ga = np.abs(dv[..., t]) + Sa
            mt, io, rh, at, vt = m[..., t], iota[..., t], rho[..., t], a[..., t], v[..., t]
            hb, Eb = before[..., t], Ebefore[..., t]
            q = np.where(vt > 0, vt / np.where(mt > 0, np.where(keep, 1, mt), 1), 0)
            k1, k2 = io * x[..., t] * at * q, hb * vt
            e = eb[..., t] + (20 + np.abs(r[..., t]) + np.abs(i[..., t])) * U
            Tk = np.where(keep, 0, at * (k1 - k2))
            eTk = np.where(keep, 0, at * ((np.abs(k1) + np.abs(k2)) * e + 2 * Eb * vt))
            T[..., t], eT[..., t] = g * Tk, eg * np.abs(Tk) + ga * eTk
            dr[..., t], edr[..., t] = g * Tk * (1 - rh), (eg * np.abs(Tk) + ga * (eTk + np.abs(Tk) * e)) * sigmoid(-r[..., t])
            ki, kx = mt * io * x[..., t] * sigmoid(-i[..., t]), mt * io
            di[..., t], edi[..., t] = g * ki, (eg + ga * e) * np.abs(ki)
            dx[..., t], edx[..., t] = g * kx, (eg + ga * e) * kx
            ns, nSg, nSa = np.where(keep, 0, at * g), np.where(keep, 0, at * (eg + (ea[..., t] + U) * ga)), np.where(keep, 0, at * ga)
            s, Sg, Sa = np.where(on, ns, s), np.where(on, nSg, Sg), np.where(on, nSa, Sa)
        dr = T * sigmoid(-r)
        out.update(dx=rounded(dx, edx), dr=rounded(dr, edr), di=rounded(di, edi))
        T, eT, dr, edr, di, edi = (np.where(inside, w, 0) for w in (T, eT, dr, edr, di, edi))
        adds = (L / 16 + 16 + B) * U  # additions on a value's way into its sum

        def total(val, err, scale=1.0, es=0.0):
            return val.sum((0, 2)) * scale, ((2 * err).sum((0, 2)) + (adds + es) * np.abs(val).sum((0, 2))) * np.abs(scale) + 1e-30

        out["dlam"] = total(T, eT, sigmoid(lam) / soft, 8 * U)
        out["dr_bias"], out["di_bias"] = total(dr, edr), total(di, edi)
        out["dinitial_state"] = (s, 2 * Sg + 1e-30)
    return out


def check(got, want, what):
    """Every element within its bound; NaN and infinity in the same places."""
    val, err = want
    got = f64(got)
    assert got.shape == val.shape, (what, got.shape, val.shape)
    assert np.array_equal(np.isnan(got), np.isnan(val)), what + ": NaN in other places"
    fine = np.isfinite(val)
    assert np.array_equal(got[~fine & ~np.isnan(val)], val[~fine & ~np.isnan(val)]), what + ": other infinities"
    over = np.abs(got[fine] - val[fine]) / err[fine]
    if over.size:
        k = int(np.argmax(over))
        assert over[k] <= 1, f"{what}: off by {over[k]:.2f} of the bound ({got[fine][k]!r}, {val[fine][k]!r}, bound {err[fine][k]!r})"
        return float(over[k])
    return 0.0
