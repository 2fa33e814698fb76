"""mla_draft_verify where the random number of the next token lies next to a border: against the
definition in rational arithmetic, at distances that 64-bit sums resolve and 32-bit ones do not."""
from fractions import Fraction

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def run(mv, p, q, tok, par, u, un):
    t = [None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in (p, q, tok, par, u, un)]
    got = [x.cpu().numpy() for x in mv.draft_verify(*t)]
    assert mv.device_status(clear=True) == 0
    return got


def after_rejections(p, q, tokens):
    """The residual R in Fractions after these tokens, drawn from q, were all rejected."""
    P, Q, S = [Fraction(float(x)) for x in p], [Fraction(float(x)) for x in q], Fraction(1)
    R = P
    for _ in tokens:
        R = [max(r - S * d, Fraction(0)) for r, d in zip(R, Q)]
        S = sum(R)
    return R


def next_token(R, un):
    """(token, distance of the nearest border)."""
    T, c, near, token = sum(R), Fraction(0), None, None
    want = Fraction(float(un)) * T
    for i, r in enumerate(R):
        c += r
        near = abs(c - want) if near is None else min(near, abs(c - want))
        if token is None and c > want:
            token = i
    return token, near


# (p, q, u_next, token): the first draft, the last token, is rejected
FOUND = [([0.625450611114502, 0.17584046721458435, 0.1987089067697525],
          [0.13722887635231018, 0.047644827514886856, 0.8151262998580933], 0.7920311093330383, 1),
         ([0.9078309535980225, 0.021481962874531746, 0.07068708539009094],
          [0.10679996758699417, 0.008726878091692924, 0.8844731450080872], 0.9843262434005737, 0)]


@pytest.mark.parametrize("p,q,un,token", FOUND)
def test_borders_within_1e_8(cuda_lib, p, q, un, token):
    p, q = np.float32([[p, p]]), np.float32([[q, q]])
    assert next_token(after_rejections(p[0, 0], q[0, 0], [2]), np.float32(un))[0] == token
    n, toks, _ = run(cuda_lib, p, q, np.int32([[0, 2]]), None, np.float32([[0, 0.9999]]), np.float32([un]))
    assert n[0] == 0 and toks[0].tolist() == [token, -1]


@pytest.mark.parametrize("rejected", [0, 1, 2, 4])
@pytest.mark.parametrize("kind", ["large", "even"])
def test_random_borders(cuda_lib, kind, rejected):
    """Rows with a border within half a step of u_next (2^-25): the leading part of a large residual is a
    tie as often as not, and every operation's error counts.  Each element of R is within one unit of
    2^-44, the normalisers S off by up to V of them move R by as much again, and so on for each
    rejection: borders nearer than that are left out (a handful in a thousand), but for those that
    u_next meets exactly.  Those come from rows whose elements are whole units, and from u_next = 0
    before elements of zero, and have to be exact, too."""
    rng = np.random.default_rng(100 * rejected + len(kind))
    B, V, q_len = 1500, 4, rejected + 2
    p, q = np.zeros((B, q_len, V), np.float32), np.zeros((B, q_len, V), np.float32)
    un, want, near = np.zeros(B, np.float32), [], []
    for b in range(B):
        if kind == "large":
            x = np.array([rng.uniform(0.55, 0.95), *rng.random(V - 1) * 0.1])
        else:
            x = rng.random(V)
        x /= x.sum()
        y = np.append(rng.random(V - 1) * 0.1, 1.0)    # the drafter's mass sits on the last token
        y /= y.sum()
        p[b], q[b] = x, y
        R = after_rejections(p[b, 0], q[b, 0], range(rejected))
        c = np.cumsum([float(r) for r in R])
        un[b] = np.float32(c[rng.integers(0, V - 1)] / c[-1])
        if un[b] >= 1:
            un[b] = np.float32(0.5)
        w, d = next_token(R, un[b])
        want.append(w)
        near.append(d)
    # siblings, all with a token that the drafter likes and the target does not: rejected
    par = np.zeros((B, q_len), np.int32)
    par[:, 1 + rejected:] = -1
    tok = np.full((B, q_len), V - 1, np.int32)
    u = np.full((B, q_len), 0.99999, np.float32)
    n, toks, _ = run(cuda_lib, p, q, tok, par, u, un)
    clear = [d == 0 or d > Fraction(4 * V * (rejected + 1), 1 << 44) for d in near]
    assert sum(clear) > 0.95 * B
    live = [b for b in range(B) if clear[b] and n[b] == 0]
    assert len(live) > 0.9 * B
    bad = [b for b in live if toks[b, 0] != want[b]]
    assert not bad, f"{len(bad)} of {len(live)}: stream {bad[0]}, token {toks[bad[0], 0]} for {want[bad[0]]}"


def test_product_with_u_next(cuda_lib):
    """Rows whose first two elements sum to the integer (in units of 2^-44) next above u_next times the
    whole, less than 2^-10 away, so that the product rounds to that integer: the second element is the
    token, since the sum up to it is greater than the product.  And rows where the two are equal: it is not."""
    rng = np.random.default_rng(7)
    unit, B = 1 << 44, 200
    p, un, want = np.zeros((B, 1, 4), np.float32), np.zeros(B, np.float32), []
    two = lambda c: (c >> 21 << 21, c & (1 << 21) - 1)          # each a float's 24 bits
    for b in range(B):
        while True:
            total = int(rng.integers(unit * 6 // 10, unit * 9 // 10))
            m = rng.integers(1 << 23, 1 << 24, 4096, dtype=np.uint64)
            if b % 2:                                           # the product is an integer
                total, m = total >> 24 << 24, m[:1]
                break
            low = (m * np.uint64(total & 0xffffff)) % np.uint64(1 << 24)     # of the product, in units of 2^-24
            m = m[low >= np.uint64((1 << 24) - (1 << 14) + 1)]
            if len(m):
                break
        m = int(m[0])
        border = -(-m * total >> 24)                            # ceil(u T)
        p[b, 0] = [Fraction(x, unit) for x in (*two(border), *two(total - border))]
        assert sum(Fraction(float(x)) for x in p[b, 0]) == Fraction(total, unit)
        un[b] = m / (1 << 24)
        want.append(next_token([Fraction(float(x)) for x in p[b, 0]], un[b])[0])
    assert want[::2] == [1] * (B // 2) and all(w >= 2 for w in want[1::2])
    zero = np.zeros((B, 1), np.int32)
    _, toks, _ = run(cuda_lib, p, None, zero, None, np.zeros((B, 1), np.float32), un)
    assert toks[:, 0].tolist() == want


def test_small_u_next(cuda_lib):
    """u_next down to the smallest float, in front of elements of zero and of one unit."""
    un = np.float32([0.0, 1e-45, 1e-40, 1.2e-38, 2.0 ** -64, 2.0 ** -63, 2.0 ** -44, 2.0 ** -43, 2.0 ** -41, 2.0 ** -24, 0.5])
    row = np.zeros(70, np.float32)
    row[[3, 5, 6, 40]] = 2.0 ** -44, 2.0 ** -43, 0.5, 0.5
    p = np.broadcast_to(row, (len(un), 1, 70)).copy()
    want = [next_token([Fraction(float(x)) for x in row], u)[0] for u in un]
    zero = np.zeros((len(un), 1), np.int32)
    _, toks, _ = run(cuda_lib, p, None, zero, None, np.zeros((len(un), 1), np.float32), un)
    assert toks[:, 0].tolist() == want and set(want) >= {3, 5, 6}
