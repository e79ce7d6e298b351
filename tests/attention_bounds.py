"""Bounds of one attention row that stay sharp for long ones (u = 2^-8 the half step of bf16, E = 2^-24 that of fp32).

A row's error before its rounding to bf16, per element:

    e = sum_j p_j |v_j| delta_j + |o| sum_j p_j delta_j + 2 c E a + 3 E |o|,        a = sum_j p_j |v_j|

delta_j bounds the relative error of weight j: the score's fp32 sum over d exact products, 2 E a term (the tensor core may
truncate), 2 d E scale sum_i |q_i k_ji|; its roundings by the scale (4 E |s_j|), by the reference maximum (at most 8 log2 units
behind the true one: E (|s_j - m| + 8)) and in the exponential (4 E). c counts the fp32 additions that follow each
other in the sums over the keys; 3 E |o| is the division. Two ways for the weights to enter the second product:

* as two bf16 values, within 2^-17 of each: another 2^-17 in delta_j. Then the result is between the roundings of
  o - e and o + e, which leaves nothing for the output's own rounding, the largest part of the error;
* as one, within u of each: sum_j p_j v_j u_j with |u_j| <= u. For long rows u a is far too much: taken as independent and
  of mean zero these roundings make a vector whose norm exceeds 6 u sqrt(sum_j p_j^2 |v_j|^2) with a probability of
  less than 2 exp(-18) = 3e-8 (Hoeffding's bound for vectors). Then the row's error is held in the norm, to
  u |o| + |e| + that.
"""
import numpy as np
import torch

U, E = 2.0 ** -8, 2.0 ** -24


def row(q, k, v, chain, scale=None, rounded=0):
    """q [d], k, v [n, d] in fp64; the first `rounded` keys' weights enter as one bf16 value. Returns o, e [d] and the norm
    that those roundings may have."""
    d = q.shape[0]
    scale = d ** -0.5 if scale is None else scale
    s = (k @ q) * scale
    p = np.exp(s - s.max())
    p /= p.sum()
    delta = 2 * d * E * scale * (np.abs(k) @ np.abs(q)) + E * (4 * np.abs(s) + np.abs(s - s.max()) + 12)
    delta[rounded:] += 2.0 ** -17
    o, a = p @ v, p @ np.abs(v)
    e = (p * delta) @ np.abs(v) + np.abs(o) * (p @ delta) + 2 * chain * E * a + 3 * E * np.abs(o)
    return o, e, 6 * U * np.sqrt((p[:rounded] ** 2) @ (v[:rounded] ** 2).sum(-1))


def rounded_within(got, o, e):
    """Whether a bf16 row is a rounding of something within e of o."""
    lo, hi = (torch.from_numpy(x).to(torch.bfloat16).double().numpy() for x in (o - e, o + e))
    return bool(((lo <= got) & (got <= hi)).all())


def norm_within(got, o, e, r):
    return bool(np.linalg.norm(got - o) <= U * np.linalg.norm(o) + np.linalg.norm(e) + r)
