"""Verification where u lies next to a border: a running sum, or a draft's acceptance, that exact arithmetic puts 2^-43 (of it) to either side.

What decides is a small rest of large numbers: p - c q of a draft near its target, 1 less the rejected drafts' probabilities.
Rounding: what is left of a token is off by 2^-47 of itself and of (c - 1) q; a sum of it by 2^-48 for each of some ten additions in
turn, in a lane, over lanes and over warps.  In random directions that is about 2^-46, an eighth of the distance."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import block_quantized_gemv_gb300 as bqg
from block_quantized_gemv_gb300 import build as bqg_build
from test_gpu_verify import verify

pytestmark = pytest.mark.gpu

NEAR = Fraction(1, 2 ** 43)
MOST = float(np.float32(1 - 2.0 ** -24))


@pytest.fixture(scope="module", autouse=True)
def built():
    bqg_build.build()


def pieces(x, n=3):
    """A positive number as n fp32 ones, each the most that fits (to 2^-24 n of it)."""
    out = []
    for _ in range(n):
        f = np.float32(float(x))
        if Fraction(float(f)) > x:
            f = np.nextafter(f, np.float32(0))
        out.append(f)
        x -= Fraction(float(f))
    return out


def solve(f, x0, x1, aim, turns=12):
    """x with f(x) = aim, nearly: f is monotone and all but linear."""
    f0, f1 = f(x0), f(x1)
    for _ in range(turns):
        if f1 == aim or f0 == f1:
            break
        x0, x1, f0 = x1, x1 + (aim - f1) * (x1 - x0) / (f1 - f0), f1
        x1 = Fraction(round(x1 * 2 ** 120), 2 ** 120)
        f1 = f(x1)
    return x1


def rests(p, q, k):
    """r and Z after each of k rejections of sampled drafts."""
    c, Z, out = Fraction(0), Fraction(1), []
    for _ in range(k):
        c += Z
        r = [max(a - c * b, Fraction(0)) for a, b in zip(p, q)]
        Z = sum(r)
        out.append((r, Z))
    return out


def call(target, draft, tokens, u, want=None):
    """One sequence: all drafts behind token 0."""
    n = len(tokens)
    t = lambda a, **kw: torch.tensor(np.asarray(a), device="cuda", **kw)
    rows = lambda x: torch.from_numpy(x)[None].expand(n, -1).contiguous()
    target, draft = rows(target), None if draft is None else rows(draft)
    parent = [-1] + [0] * (n - 1)
    got = bqg.tree_verify(target.cuda(), t(tokens, dtype=torch.int32), t([0, n], dtype=torch.int32), n, t(u, dtype=torch.float32),
                          parent=t(parent, dtype=torch.int32), draft=None if draft is None else draft.cuda())
    if want is None:
        want = verify(target, tokens, [n], u, parent, draft, n)
    assert tuple(x.tolist() for x in got) == want
    return want


def near_target(V, seed, apart):
    """A draft `apart` from its target, with three last tokens that it never draws (to tune with), and tokens it draws too often."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=V) * 2
    p = (np.exp(x) / np.exp(x).sum()).astype(np.float32)
    q = (p.astype(np.float64) * (1 + apart * rng.normal(size=V))).astype(np.float32)
    p[-3:], q[-3:] = 0, 0
    often = [int(i) for i in np.argsort(-p) if q[i] > np.float64(p[i]) * (1 + apart / 4)][:8]
    return p, q, often


@pytest.mark.parametrize("apart", [1e-2, 1e-4, 1e-6])
@pytest.mark.parametrize("k", [1, 2, 3, 5])
@pytest.mark.parametrize("side", [-1, 1])
def test_next_token_after_rejections(apart, k, side):
    p, q, often = near_target(1501, k, apart)
    P, Q = [Fraction(float(x)) for x in p], [Fraction(float(x)) for x in q]
    r, Z = rests(P, Q, k)[-1]
    # the first token at which the running sum is past a half of it, but for what is tuned
    run, x = Fraction(0), -1
    while run * 2 <= Z:
        x += 1
        run += r[x]

    def beyond(tau):                                                          # the running sum less its half, of the whole
        r, Z = rests(P[:-1] + [tau], Q, k)[-1]
        return (sum(r[:x + 1]) - Z / 2) / Z

    tau = solve(beyond, Fraction(0), Z / 1000, side * NEAR)
    assert tau > 0
    p[-3:] = pieces(tau)
    exact = beyond(sum(Fraction(float(v)) for v in p[-3:]))
    assert abs(exact / (side * NEAR) - 1) < 0.1
    want = call(p, q, [0] + often[:k], [0.5] + [MOST] * k)
    assert want[0] == [1] and (want[2][0] == x) == (side > 0)


@pytest.mark.parametrize("apart", [1e-2, 1e-4, 1e-6])
@pytest.mark.parametrize("k", [1, 2, 4])
@pytest.mark.parametrize("side", [-1, 1])
def test_acceptance_after_rejections(apart, k, side):
    p, q, often = near_target(1501, 10 + k, apart)
    P, Q = [Fraction(float(x)) for x in p], [Fraction(float(x)) for x in q]
    c = 1 + sum(Z for _, Z in rests(P, Q, k)[:-1])
    Z = rests(P, Q, k)[-1][1]
    at = int(np.argsort(-p)[20])

    def beyond(tau):                                                          # what is left of the draft less u q Z, of the latter
        r, Z = rests(P[:at] + [first] + P[at + 1:-1] + [tau], Q, k)[-1]
        border = Q[at] * Z / 2
        return (first - (1 + sum(z for _, z in rests(P[:at] + [first] + P[at + 1:-1] + [tau], Q, k)[:-1])) * Q[at] - border) / border

    # a probability a little above the border, which tau, by the sums that it enters, raises to it
    first = Fraction(float(np.nextafter(np.nextafter(np.float32(float((c + Z / 2) * Q[at])), np.float32(1)), np.float32(1))))
    for i in range(20):
        if beyond(Fraction(0)) > 0:
            break
        first = Fraction(float(np.float32(float(first) * (1 + 2.0 ** (i - 23)))))
    tau = solve(beyond, Fraction(0), Z / 1000, side * NEAR)
    assert tau > 0
    p[at], p[-3:] = np.float32(float(first)), pieces(tau)
    exact = beyond(sum(Fraction(float(v)) for v in p[-3:]))
    assert abs(exact / (side * NEAR) - 1) < 0.1
    want = call(p, q, [0] + often[:k] + [at], [0.25] + [MOST] * k + [0.5])
    assert want[0] == [2 if side > 0 else 1]


@pytest.mark.parametrize("side", [-1, 1])
def test_acceptance_of_a_chosen_draft_after_rejections(side):
    """Small probabilities are rejected before the large ones: their last bits are what is left at the end."""
    V = 300
    rng = np.random.default_rng(3)
    p = np.zeros(V, dtype=np.float32)
    p[:4] = (rng.random(4) + 1).astype(np.float32) * np.float32(1e-9)
    p[4], p[5] = np.float32(0.6123456), np.float32(0.3876382)
    left = 1 - sum(Fraction(float(x)) for x in p[:6])
    assert 0 < left < 2e-5
    p[6] = np.float32(float(left / 4))                                        # the draft at the border: 2 p = Z
    gap = left - 2 * Fraction(float(p[6])) * (1 - side * NEAR)                # more to reject, in three pieces
    assert gap > 0
    p[7:10] = pieces(gap)
    tokens = [0, 9, 8, 0, 1, 2, 3, 7, 4, 5, 6]
    u = [0.25] + [MOST] * 9 + [0.5]
    left = 1 - sum(Fraction(float(p[t])) for t in tokens[1:-1] if t) - Fraction(float(p[0]))
    exact = Fraction(float(p[6])) / (left / 2) - 1
    assert abs(exact / (side * NEAR) - 1) < 0.1
    p[200] = np.float32(float(left / 2))
    want = call(p, None, tokens, u)
    assert want[0] == [2 if side > 0 else 1]


@pytest.mark.parametrize("V", [131075, 1 << 22, 1 << 24])
@pytest.mark.parametrize("side", [-1, 1])
def test_next_token_of_a_long_row_beside_a_large_probability(V, side):
    """A lane adds its part of the row to one large number.  At 2^24 tokens that is 128 additions one after the other, each off by
    2^-48 of it at most: 2^-45 in random directions, and the border is put 2^-42 away."""
    near = NEAR * 2 if V == 1 << 24 else NEAR
    rng = np.random.default_rng(V % 1000)
    tail = rng.random(V) * 0.1 / V * 2
    p = tail.astype(np.float32)
    p[0] = np.float32(0.9123456)
    p[-3:] = 0
    unit = 60
    whole = np.round(p.astype(np.float64) * 2.0 ** unit).astype(np.int64)     # exact where a value is a multiple of 2^-60
    p = (whole.astype(np.float64) * 2.0 ** -unit).astype(np.float32)
    whole = (p.astype(np.float64) * 2.0 ** unit).astype(np.int64)
    assert (whole.astype(np.float64) * 2.0 ** -unit == p).all()
    total, run = sum(int(x) for x in np.add.reduceat(whole, np.arange(0, V, 4096))), np.cumsum(whole)
    u = float(np.float32(0.96))
    x = int(np.searchsorted(run, int(Fraction(u) * total), side="right"))
    over = int(run[x]) - Fraction(u) * total
    # over - u tau = +- near of the whole
    tau = (over - side * near * total) / Fraction(u) / 2 ** unit
    assert tau > 0
    p[-3:] = pieces(tau)
    t = sum(Fraction(float(v)) for v in p[-3:])
    exact = (Fraction(int(run[x]), 2 ** unit) - Fraction(u) * (Fraction(total, 2 ** unit) + t)) / Fraction(total, 2 ** unit)
    assert abs(exact / (side * near) - 1) < 0.1
    nxt = x if side > 0 else x + 1 + int(np.argmax(p[x + 1:] > 0))
    call(p, None, [0], [u], want=([1], [[0]], [nxt]))
