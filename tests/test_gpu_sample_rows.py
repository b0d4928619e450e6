"""Sampling of rows that several CTAs share, or that take the long ways through the kernel, against the
plain 64-bit form (tests/serve_ref.py)."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import serve_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def body(rows, V, dtype, seed, scale, peaks):
    """Rows of a Gaussian body, with `peaks` likely tokens at falling scores."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, V, generator=g, device="cuda") * scale
    if peaks:
        at = torch.rand(rows, peaks, generator=g, device="cuda").argsort(1) * (V // peaks)
        x.scatter_(1, at, 14.0 - 1.7 * torch.log1p(torch.arange(peaks, device="cuda").float()).expand(rows, peaks))
    return x.to(dtype), torch.rand(rows, generator=g, device="cuda")


def check(x, u, sets, take, probs=True):
    """Draws all rows (they decide how many CTAs share one) with row r's settings sets[r % len(sets)] and
    holds rows `take` to the plain form."""
    from block_diffusion_drafter_forward_gb300 import sample
    rows = x.shape[0]
    col = [[sets[r % len(sets)][i] for r in range(rows)] for i in range(4)]
    T, p, lo = (torch.tensor(col[i], dtype=torch.float32, device="cuda") for i in (0, 2, 3))
    k = torch.tensor(col[1], dtype=torch.int32, device="cuda")
    pr = torch.empty(rows, device="cuda") if probs else None
    got = sample(x, u, T, k, p, lo, probs=pr)
    tokens = (got[0] if probs else got).tolist()
    for r in take:
        T_, p_, lo_, u_ = (float(v[r]) for v in (T, p, lo, u))
        want, wp = R.sample(x[r].double().cpu().numpy(), u_, T_, col[1][r], p_, lo_)
        assert tokens[r] == want, (r, tokens[r], want, T_, col[1][r], p_, lo_, u_)
        if probs:
            assert abs(float(pr[r]) - wp) <= 2.0 ** -23 * wp + 1e-12, (r, float(pr[r]), wp)


# (vocabulary, type, rows): CTAs of a row have unequal numbers of blocks, so that a share of the row
# counted by each for itself sent some of them by one floor and the others by another
UNEVEN = [(262144, torch.bfloat16, 1), (262144, torch.bfloat16, 16), (262144, torch.bfloat16, 100), (262144, torch.bfloat16, 200),
          (262144, torch.float32, 16), (262144, torch.float32, 64), (131072, torch.bfloat16, 100), (131072, torch.float32, 20),
          (163840, torch.bfloat16, 90), (102400, torch.float32, 90), (49152, torch.bfloat16, 200)]


@pytest.mark.parametrize("V,dtype,rows", UNEVEN)
def test_every_cta_of_a_row_goes_by_one_floor(V, dtype, rows):
    k_sets = [(0.9, k, p, 0.0) for k, p in ((400, 1.0), (450, 0.9), (600, 1.0), (868, 1.0), (900, 0.95), (1000, 0.8), (1000, 1.0), (1095, 1.0),
                                            (1300, 0.99), (1800, 1.0), (2000, 1.0), (2100, 0.9))]
    p_sets = [(1.0, 0, 0.95, 0.0), (0.8, 0, 0.9, 0.0), (1.2, 0, 0.99, 0.0), (2.0, 0, 0.9, 0.0), (0.6, 0, 0.999, 0.0), (1.0, 0, 0.5, 0.01)]
    for seed, (scale, peaks) in enumerate(((2.0, 48), (1.0, 0))):
        x, u = body(rows, V, dtype, seed, scale, peaks)
        for sets in (k_sets, p_sets):
            if rows == 1:
                for s in sets[::2]:
                    check(x, u, [s], [0])
            else:
                check(x, u, sets, list(range(0, min(rows, len(sets)), 1 + seed)) + [rows - 1])


# (vocabulary, rows): one CTA of a row, two, and eight
@pytest.mark.parametrize("V,rows", [(20000, 460), (40000, 8), (151936, 8)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_runs_of_nan_are_no_candidates(V, rows, dtype):
    """NaN logits count as -inf, also where a thread meets nothing else; the largest logit in the run's
    slice, ahead of it, behind it and elsewhere."""
    sets = [(1.0, 0, 1.0, 0.0), (0.0, 0, 1.0, 0.0), (0.8, 50, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.05), (1.0, 700, 0.95, 0.01),
            (1.5, 0, 0.99, 0.0), (3.0, 0, 0.9, 0.0)]
    x, u = body(rows, V, dtype, V, 2.0, 16)
    runs = [(V // 2, V), (V // 2, V // 2 + 5000), (0, V // 3), (V // 3, V - 3), (3, V - 1), (V - 4000, V - 500), (V // 2 - 2100, V // 2 + 2100), (8, 1500)]
    for r in range(rows):
        a, b = runs[r % len(runs)]
        x[r, a:b] = float("nan")
        x[r, (a - 1, min(b, V - 1))[r // 8 % 2]] = 16.0 if a else -1.0
    for shift in (0, 1, 3) if rows == 8 else (0,):
        take = range(16) if rows > 8 else range(8)
        check(x, u, sets[shift:] + sets[:shift], take)


def equal_tail(c, N, p, u):
    """(kept tail, token, distances) of a row that holds 0 and then N logits c < 0, at T = 1, exactly: the
    distances of p and u from the borders next to them, in parts of the row's mass."""
    w = Fraction(float(np.exp(np.float64(c))))
    total = 1 + N * w
    n = N
    dp = Fraction(1)
    if p < 1:
        at = (Fraction(p) * total - 1) / w
        n = max(0, min(N, math.ceil(at)))
        dp = abs(at - round(at)) * w / total
    kept = 1 + n * w
    at = (Fraction(u) * kept - 1) / w
    token = 0 if at < 0 else 1 + min(n - 1, math.floor(at))
    return n, token, float(dp), float(abs(at - round(at)) * w / kept)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("top_k", [0, 230000])
def test_long_prefixes_at_their_borders(top_k, dtype):
    """One likely token and a tail of equal ones, whose number kept the token at u near 1 tells: p 2e-11 to
    4e-10 of the mass from a border (the definition leaves 1e-11 open), which the tail's common rounding
    must not cross."""
    V, rows = 262144, 64
    N = top_k - 1 if top_k else V - 1
    rng = np.random.default_rng(7)
    x = torch.empty(rows, V)
    ps, us, want = [], [], []
    for r in range(rows):
        c = -17.0 - 0.125 * (r % 16)
        x[r] = c
        x[r, 0] = 0.0
        tail = float(N * np.exp(c) / (1 + N * np.exp(c)))
        while True:
            p = float(np.float32(1 - tail * rng.uniform(0.2, 0.9)))
            if 2e-11 < equal_tail(c, N, p, 0.5)[2] < 4e-10:
                break
        u = 1.0
        while True:
            u = float(np.nextafter(np.float32(u), np.float32(0)))
            n, token, _, du = equal_tail(c, N, p, u)
            if du > 1e-9:
                break
        ps.append(p), us.append(u), want.append(token)
    from block_diffusion_drafter_forward_gb300 import sample
    k = torch.full((rows,), top_k, dtype=torch.int32, device="cuda") if top_k else None
    got = sample(x.to(dtype).cuda(), torch.tensor(us, device="cuda"), None, k, torch.tensor(ps, device="cuda"))
    assert got.tolist() == want


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [8, 230])
def test_u_at_the_borders_of_a_flat_tail(rows, dtype):
    """Temperature alone over the same rows: u 2e-11 to 4e-10 of the mass from a border."""
    V = 262144
    rng = np.random.default_rng(8)
    x = torch.empty(rows, V, dtype=dtype, device="cuda")
    us, want = [], []
    for r in range(rows):
        c = -14.0 - 0.0625 * (r % 32)
        x[r] = c
        x[r, 0] = 0.0
        tail = float((V - 1) * np.exp(c) / (1 + (V - 1) * np.exp(c)))
        while True:
            u = float(np.float32(1 - tail * rng.uniform(0.01, 0.99)))
            _, token, _, du = equal_tail(c, V - 1, 1.0, u)
            if 2e-11 < du < 4e-10:
                break
        us.append(u), want.append(token)
    from block_diffusion_drafter_forward_gb300 import sample
    u = torch.tensor(us, device="cuda")
    assert sample(x, u).tolist() == want
    assert sample(x, u, probs=torch.empty(rows, device="cuda"))[0].tolist() == want


def late_maximum(V, dtype, a, b, mid=0):
    """Rows whose maximum (1) comes late: against the maximum until then (0, at 5000) the body's weights are
    above 2^-40, against the row's they are below and count as 0.  a, b: the two logits behind the maximum."""
    x = torch.full((len(a), V), -27.0)
    if mid:
        x[:, 7:V - 4000:V // mid] = -12.0
    x[:, 5000] = 0.0
    at = [V - 2712, V - 1644, V - 644]
    x[:, at[0]], x[:, at[1]], x[:, at[2]] = 1.0, torch.tensor(a).float(), torch.tensor(b).float()
    return x.to(dtype).cuda(), at


@pytest.mark.parametrize("rows", [8, 230])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_row_has_a_token_at_the_ends_of_u(rows, dtype):
    """u = 0 and u = 1: the first and the last logit that counts, where whole stretches ahead and behind count
    as 0 only since the row's maximum is known."""
    from block_diffusion_drafter_forward_gb300 import sample
    x, at = late_maximum(262144, dtype, [0.25] * rows, [-0.5] * rows)
    for u, want in ((0.0, 5000), (1.0, at[2])):
        tokens = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
        probs = torch.full((rows,), -7.0, device="cuda")
        us = torch.full((rows,), u, device="cuda")
        assert sample(x, us, tokens=tokens).tolist() == [want] * rows
        tokens.fill_(-7)
        sample(x, us, tokens=tokens, probs=probs)
        assert tokens.tolist() == [want] * rows and bool((probs > 0).all())


def near_border(rows, seed, other, of, step):
    """Logits a > b > 0 (multiples of 1/128) and an fp32 fraction f of the row's mass 1 + e^-1 + e^(a-1) +
    e^(b-1) + `other`, next to the border of(a, b) in direction `step` and so near that a body of
    262144 e^-28, counted, would move the border past it."""
    rng, out = np.random.default_rng(seed), []
    while len(out) < rows:
        b, a = sorted(rng.integers(1, 64, 2) / 128.0)
        if a == b:
            continue
        total = 1 + math.exp(-1) + math.exp(a - 1) + math.exp(b - 1) + other
        ahead = of(a, b)
        f = np.float32(ahead / total)
        if (float(f) * total - ahead) * step <= 0:
            f = np.nextafter(f, np.float32(step > 0))
        d = abs(float(f) * total - ahead)
        body = 262144 * math.exp(-28.0) * (1 - float(f) if step > 0 else float(f))
        if 1e-9 < d < 0.8 * body:
            out.append((a, b, float(f)))
    return [list(v) for v in zip(*out)]


@pytest.mark.parametrize("rows", [8, 230])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_weights_below_the_cut_move_no_border(rows, dtype):
    """The body of such a row, 1.8e-7 of the mass were it counted, moves neither u's border between a and b
    (u lies just above it: b) nor p's behind a (p lies just below it: b goes)."""
    from block_diffusion_drafter_forward_gb300 import sample
    V, e = 262144, math.exp
    a, b, u = near_border(rows, 2, 0.0, lambda a, b: e(-1) + 1 + e(a - 1), 1)
    x, at = late_maximum(V, dtype, a, b)
    assert sample(x, torch.tensor(u, device="cuda")).tolist() == [at[2]] * rows
    mid = len(range(7, V - 4000, V // 1500))
    a, b, p = near_border(rows, 3, mid * e(-13.0), lambda a, b: 1 + e(a - 1), -1)
    x, at = late_maximum(V, dtype, a, b, 1500)
    last = torch.full((rows,), 1 - 2.0 ** -24, device="cuda")
    assert sample(x, last, top_p=torch.tensor(p, device="cuda")).tolist() == [at[1]] * rows
