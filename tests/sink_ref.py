"""Plain 64-bit attention with a sliding window and sink tokens, with the error
each output may have, derived from the roundings the operators make.

Half a step of bf16 is h = 2^-8 relative. The operators form the weights P in
fp32 and round them to bf16 for the products, so
  |out error| <= h sum_s P |v|  +  h |out|                    (P, then out itself)
  |dv  error| <= h sum_p P |dO| [+ h |dv| for bf16 gradients]
dS = P (dP - delta) is rounded to bf16, and delta is taken from the rounded out,
off by at most sum_d |dO| |out error|:
  |dS  error| <= h |dS| + P (delta error)
  |dq  error| <= scale sum_s |dS error| |k|, |dk error| <= scale sum_p |dS error| |q|
[+ h of the value]. What fp32 adds (products of bf16 are exact, sums of at most a
few thousand terms at 2^-23 of the terms' magnitudes, exponentials at 2^-22) is
covered by SLACK relative to the same sums of magnitudes. Those are bounds for
every element; over a whole tensor the roundings do not all point the same way,
so the root mean square is held to the root of the summed squares."""
from __future__ import annotations

import math

import torch

import oracle

H = 2.0 ** -8
SLACK = 1e-4
LSE_ABS = 2e-4  # scores: up to 512 products, |q.k| scale about 10: 512 * 2^-23 * 10 < 1e-4 twice


def visible(doc: torch.Tensor, row_offset: int, L: int, kv_offset: int, S_kv: int, window: int, n_sink: int):
    """[B, L, S_kv] bool from the rule, position by position."""
    B, S = doc.shape
    start = torch.zeros_like(doc)
    for b in range(B):
        at = 0
        for s in range(S):
            if s and doc[b, s] != doc[b, s - 1]:
                at = s
            start[b, s] = at
    p = torch.arange(row_offset, row_offset + L)[None, :, None]
    s = torch.arange(kv_offset, kv_offset + S_kv)[None, None, :]
    dp, ds = doc[:, row_offset:row_offset + L, None], doc[:, None, kv_offset:kv_offset + S_kv]
    st = start[:, None, kv_offset:kv_offset + S_kv]
    ok = (dp == ds) & (dp != 0) & (s <= p)
    if window > 0:
        ok &= (p - s < window) | (s - st < n_sink)
    return ok


def reference(c: dict, n_sink: int, og=None) -> dict:
    """Values and bounds ("out", "e_out", ...) of the case's shard; `og`: the oracle's geometry, for dropout."""
    w = c["w"]
    doc = torch.from_numpy(c["doc"]).long()
    ok = visible(doc, c["row_offset"], w.L, c["kv_offset"], c["S_kv"], c["window"], n_sink)
    q, k, v, do = (c[n].double() for n in ("q", "k", "v", "do"))
    G, scale = w.G, float(w.D) ** -0.5
    r = {n: torch.zeros(w.B, w.Hq, w.L, w.D, dtype=torch.float64) for n in ("out", "e_out", "r_out", "dq", "e_dq", "r_dq")}
    r.update({n: torch.zeros(w.B, w.Hkv, c["S_kv"], w.D, dtype=torch.float64)
              for n in ("dk", "e_dk", "r_dk", "dv", "e_dv", "r_dv")})
    r["lse"] = torch.full((w.B, w.Hq, w.L), -math.inf, dtype=torch.float64)
    for b in range(w.B):
        for h in range(w.Hq):
            hk = h // G
            x = (q[b, h] @ k[b, hk].T * scale).masked_fill(~ok[b], -math.inf)
            lse = torch.logsumexp(x, 1)
            p = torch.exp(x - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None])
            z = torch.ones_like(p)
            if og is not None and og.dropout_p > 0:
                z = torch.from_numpy(oracle.dropout_factors(og, b, h))
            pz = p * z
            out = pz @ v[b, hk]
            e_out = (H + SLACK) * (pz @ v[b, hk].abs()) + H * out.abs()
            dp = z * (do[b, h] @ v[b, hk].T)
            delta = (do[b, h] * out).sum(1, keepdim=True)
            e_delta = (do[b, h].abs() * e_out).sum(1, keepdim=True)
            r_out2 = H ** 2 * (pz ** 2 @ v[b, hk] ** 2 + out ** 2)
            r_delta2 = (do[b, h] ** 2 * r_out2).sum(1, keepdim=True)
            ds = p * (dp - delta)
            mag = p * (z * (do[b, h].abs() @ v[b, hk].abs().T) + (do[b, h].abs() * out.abs()).sum(1, keepdim=True))
            e_ds = H * ds.abs() + p * e_delta + SLACK * mag
            r["lse"][b, h], r["out"][b, h], r["e_out"][b, h], r["r_out"][b, h] = lse, out, e_out, r_out2
            r["dq"][b, h] = scale * ds @ k[b, hk]
            r["e_dq"][b, h] = scale * e_ds @ k[b, hk].abs()
            r["dk"][b, hk] += scale * ds.T @ q[b, h]
            r["e_dk"][b, hk] += scale * e_ds.T @ q[b, h].abs()
            r["dv"][b, hk] += pz.T @ do[b, h]
            r["e_dv"][b, hk] += (H + SLACK) * (pz.T @ do[b, h].abs())
            r["r_dq"][b, h] = scale ** 2 * ((H * ds) ** 2 @ k[b, hk] ** 2 + r_delta2 * (p @ k[b, hk]) ** 2)
            r["r_dk"][b, hk] += scale ** 2 * ((H * ds) ** 2 + p ** 2 * r_delta2).T @ q[b, h] ** 2
            r["r_dv"][b, hk] += (H * pz).T ** 2 @ do[b, h] ** 2
    return r


def check(name: str, got: torch.Tensor, ref: dict, key: str, rounded: bool):
    """`rounded`: the value itself is bf16 (out's own rounding is in its bound)."""
    d = got.detach().double().cpu()
    want, e, r2 = ref[key], ref["e_" + key], ref["r_" + key]
    assert d.shape == want.shape, (name, d.shape, want.shape)
    assert torch.isfinite(d).all(), f"{name}: not finite"
    if rounded and key != "out":
        e, r2 = e + H * want.abs(), r2 + (H * want) ** 2
    err = (d - want).abs()
    over = err - e - 1e-7
    i = int(over.argmax())
    assert over.max() <= 0, (f"{name}: error {err.flatten()[i]:.3e}, bound {e.flatten()[i]:.3e} at "
                             f"{tuple(int(x) for x in torch.unravel_index(torch.tensor(i), err.shape))}")
    rms, lim = err.pow(2).mean().sqrt(), r2.mean().sqrt() + SLACK * want.pow(2).mean().sqrt() + 1e-7
    assert rms <= lim, f"{name}: rms error {rms:.3e}, bound {lim:.3e}"


def check_lse(name: str, got: torch.Tensor, ref: dict):
    d, want = got.double().cpu(), ref["lse"]
    none = torch.isinf(want)
    assert torch.equal(d[none], want[none]), f"{name}: rows without a key"
    assert torch.isfinite(d[~none]).all()
    if (~none).any():
        err = (d - want)[~none].abs().max()
        assert err <= LSE_ABS, f"{name}: lse error {err:.3e}"
