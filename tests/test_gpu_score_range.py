"""Scores at the ends of binary32. A finite logit whose quotient x / T is past
the largest binary32 number scores +inf, as a +inf logit does, and equal scores
go to the lowest index; quotients that are huge and finite swallow their Gumbel
noise, and the largest of them wins."""
import numpy as np
import pytest

import token_sampling_logits_gb300 as gs
import workloads as W
from tests.gpu_util import to_device

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

TYPES = {W.F32: torch.float32, W.BF16: torch.bfloat16, W.F16: torch.float16}
SHAPES = [(1, 60000), (4, 3000), (80, 5001), (160, 40000), (300, 3000)]


def lowest_best(x, T):
    """The lowest index of the largest binary32 quotient; for rows whose best
    quotients are infinite, or so large that no Gumbel value (at most 16.7)
    moves them, that is the draw."""
    with np.errstate(over="ignore", invalid="ignore"):
        q = x.astype(np.float32) / np.float32(T)
    q = np.where(np.isnan(q), np.float32(-np.inf), q)
    best = q.max(1)
    assert (best > 2.0 ** 30).all()  # half a step is 32 and more: adding 16.7 changes nothing
    return np.argmax(q, 1)


def placed(x, dtype, pitch, shift):
    B, V = x.shape
    buf = torch.zeros(B * (V + pitch) + shift + 8, dtype=TYPES[dtype], device="cuda")
    view = buf[shift:shift + B * (V + pitch)].view(B, V + pitch)[:, :V]
    view.copy_(torch.from_numpy(x))
    return view


def check(x, dtype, T, **kw):
    """x: values of the type. Plain and constrained draws, rows on 16 bytes and
    off them; the list kernel and the bounds of touched elements take part
    through biases of zero."""
    B, V = x.shape
    want = lowest_best(x, T)
    state = gs.new_logit_state(B, V)
    g = torch.Generator("cuda").manual_seed(V)
    n = 40
    gs.bias_set(state, torch.randint(0, V, (B * n,), generator=g, device="cuda"),
                torch.zeros(B * n, device="cuda"),
                offsets=torch.arange(B + 1, device="cuda") * n)
    mask = torch.full((B, (V + 31) // 32), -1, dtype=torch.int32, device="cuda")
    seed = torch.arange(B, device="cuda") * 7 + 1
    offset = torch.full((B,), 3, dtype=torch.int64, device="cuda")
    t = torch.full((B,), T, device="cuda")
    for pitch, shift in (((-V) % 64, 0), (3, 1)):
        y = placed(x, dtype, pitch, shift)
        for name, got in (
                ("plain", gs.gumbel_argmax(y, t, seed, offset)),
                ("state", gs.constrained_gumbel_argmax(y, t, seed, offset, state=state)),
                ("mask", gs.constrained_gumbel_argmax(y, t, seed, offset, state=state, mask=mask))):
            got = got.cpu().numpy()
            bad = np.nonzero(got != want)[0]
            assert bad.size == 0, (name, pitch, len(bad), bad[:5], got[bad[:5]], want[bad[:5]])


@pytest.mark.parametrize("T", [1.2e-38, 2.0 ** -149, 1e-42])
@pytest.mark.parametrize("dtype", [W.F32, W.BF16, W.F16])
@pytest.mark.parametrize("B,V", SHAPES)
def test_quotients_that_overflow_tie(B, V, dtype, T):
    rng = np.random.default_rng([B, V, dtype])
    x = W.roundtrip((rng.standard_normal((B, V)) * 4).astype(np.float32), dtype)
    x[rng.random((B, V)) < 0.3] = -np.inf
    x[0, :] = -1.0  # one row with a single infinite score
    x[0, V // 2] = 6.0
    check(x, dtype, T)


@pytest.mark.parametrize("T", [0.7, 1.0 - 2.0 ** -24, 1e-3, 1e-19])
@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
@pytest.mark.parametrize("B,V", SHAPES)
def test_large_logits_that_overflow_tie(B, V, dtype, T):
    """A few logits of the last octave before the quotient overflows and the
    first after it."""
    rng = np.random.default_rng([B, V, dtype, 1])
    x = (rng.standard_normal((B, V)) * 4).astype(np.float32)
    edge, most = 3.4028234e38 * T, 3.4028234e38 if dtype == W.F32 else 3.3895e38
    some = rng.random((B, V)) < 0.01
    x[some] = np.minimum(edge * rng.uniform(0.5, 2.0, some.sum()), most)
    x[:, 1000 % V] = min(edge * 0.99999, most)
    check(W.roundtrip(x, dtype), dtype, T)


@pytest.mark.parametrize("dtype", [W.F32, W.BF16, W.F16])
def test_infinite_logits_and_overflowing_ones_tie(dtype):
    rng = np.random.default_rng(5)
    x = W.roundtrip(rng.standard_normal((100, 6000)).astype(np.float32), dtype)
    x[np.arange(100), rng.integers(0, 6000, 100)] = np.inf
    x[np.arange(50), rng.integers(0, 6000, 50)] = 30.0
    check(x, dtype, 2.0 ** -126)


@pytest.mark.parametrize("T", [1.0, 3.0, 0.25])
@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
@pytest.mark.parametrize("B,V", SHAPES)
def test_huge_finite_scores(B, V, dtype, T):
    """Scores past 2^127, where the bound's exponent leaves binary32: rising
    along the row, so that a better one follows every candidate, and falling."""
    rng = np.random.default_rng([B, V, dtype, 2])
    x = (rng.standard_normal((B, V)) * 4).astype(np.float32)
    top = 3.38e38 * min(1.0, T)
    at = np.sort(rng.choice(V, 40, replace=False))
    ramp = (top * np.linspace(0.3, 1.0, 40)).astype(np.float32)
    x[:, at] = ramp
    x[::2, at] = ramp[::-1]
    x[1::4, at[-1]] = x[1::4, at[-2]]  # the best twice: the lower index
    check(W.roundtrip(x, dtype), dtype, T)
