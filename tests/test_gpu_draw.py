"""The draw from a filter set with given random numbers and the verification of
drafts on the GPU, against their definitions in 64 bits (tests/draw_util.py).
Indices are equal except where a decision lies within draw_util.tolerance(V) of
a border; log-probabilities are within half a binary32 step and the weights'
bound."""
import math

import numpy as np
import pytest

import token_sampling_logits_gb300 as gs
from tests import draw_util as du

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def logits(rng, B, V, dtype, sd=3.0, pitch=0, shift=0):
    """[B, V] on the GPU with `pitch` elements between rows, starting `shift`
    elements into the buffer; and the same values on the host."""
    x = torch.from_numpy((rng.standard_normal((B, V)) * sd).astype(np.float32))
    buf = torch.full((B * (V + pitch) + shift,), float("nan"), dtype=TYPES[dtype], device="cuda")
    view = buf[shift:].view(B, V + pitch)[:, :V]
    view.copy_(x.cuda())
    return view, view.float().cpu().numpy()


def settings(rng, B, greedy=0.1):
    T = rng.uniform(0.3, 2.0, B).astype(np.float32)
    T[rng.random(B) < greedy] = rng.choice([0.0, -1.0, np.nan])
    k = np.where(rng.random(B) < 0.5, rng.integers(1, 200, B), rng.choice([0, -5])).astype(np.int32)
    p = np.where(rng.random(B) < 0.6, rng.uniform(0.02, 0.999, B), rng.choice([1.0, 2.0, np.nan]))
    m = np.where(rng.random(B) < 0.4, 10 ** rng.uniform(-6, 0, B), rng.choice([0.0, -1.0, np.nan]))
    return T, k, p.astype(np.float32), m.astype(np.float32)


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def check_rows(x, T, u, k, p, m, idx, lp, tol=None):
    B, V = x.shape
    tol = du.tolerance(V) if tol is None else tol
    near = 0
    for b in range(B):
        args = (0 if k is None else k[b], 1.0 if p is None else p[b], 0.0 if m is None else m[b])
        i, l, gap = du.draw(x[b], T[b], u[b], *args)
        if gap <= tol:
            near += 1
            continue
        assert idx[b] == i, (b, idx[b], i, gap, T[b], u[b], args)
        if lp is not None:
            # one rounding of the logarithm, and the weights' own error. Without a
            # filter the row's mass S may be a bounded S' with |S' - S| <= 2^-24 S (the
            # kernel takes it on that condition), and |ln(S' / S)| <= 2^-24 (1 + 2^-24).
            free = not (args[0] >= 1 or args[1] < 1 or args[2] > 0)
            most = abs(l) * 2.0 ** -24 + 2 * tol + (2.0 ** -24 * (1 + 2.0 ** -24) if free else 0)
            assert lp[b] == l or abs(lp[b] - l) <= most, (b, lp[b], l)
    assert near <= max(1, B // 50), near


def draw(x, T, u, k=None, p=None, m=None):
    idx, lp = gs.filtered_categorical(x, dev(T), dev(u), top_k=dev(k), top_p=dev(p), min_p=dev(m),
                                      logprob=True)
    return idx.cpu().numpy(), lp.cpu().numpy()


# ---- weights --------------------------------------------------------------------
@pytest.mark.parametrize("M,T", [(0.0, 1.0), (19.37, 0.7), (-3.25, 2.5), (11.0, 0.01), (1000.5, 1.0),
                                 (1e30, 1e28), (-2e-38, 1e-38), (5.0, 1e30), (7.0, math.inf),
                                 (40.0, 1e-20)])
def test_weights(M, T):
    """Each within 2^-39 of itself and half a unit of exp((x - M) / T), up to one
    factor for all; zero for -inf, NaN and what lies below half a unit."""
    M, T = np.float32(M), np.float32(T)
    rng = np.random.default_rng(5)
    z = np.concatenate([np.linspace(0, 45, 20001), rng.uniform(0, 1, 5000), [0.0, 60.0, 1e6]])
    with np.errstate(over="ignore"):
        x = (np.float64(M) - z * min(float(T), 1e30)).astype(np.float32)
    x = np.minimum(x, M)
    x = np.concatenate([x, rng.uniform(-1e-6, 0, 1000).astype(np.float32) + np.minimum(M, 0),
                        np.float32([-np.inf, np.nan, -3.4e38])])
    x = np.where(x > M, M, x).astype(np.float32)
    w = gs.debug_weights(torch.from_numpy(x).cuda(), float(M), float(T)).cpu().numpy()
    assert w[-3] == 0 and w[-2] == 0
    ok = np.isfinite(x)
    with np.errstate(over="ignore"):
        e = np.exp((x[ok].astype(np.float64) - float(M)) / max(float(T), 2.0 ** -126))
    w = w[ok].astype(np.float64) * 2.0 ** -44
    scale = w[np.argmax(x[ok])]
    assert abs(scale - 1) < 0.002
    # the reference's own argument is rounded to 2^-53 of itself
    assert (np.abs(w / scale - e) <= e * (2.0 ** -38 + 2.0 ** -46) + 2.0 ** -44).all()


# ---- the draw -------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V,B,pitch,shift", [(1, 5, 0, 0), (2, 9, 0, 0), (7, 16, 1, 0), (31, 8, 0, 3),
                                             (257, 40, 3, 1), (1000, 33, 24, 0), (4099, 24, 0, 0),
                                             (32768, 12, 0, 0), (100003, 6, 5, 0), (262144, 4, 0, 0)])
def test_draw(dtype, V, B, pitch, shift):
    rng = np.random.default_rng(V + B)
    x, h = logits(rng, B, V, dtype, pitch=pitch, shift=shift)
    T, k, p, m = settings(rng, B)
    u = rng.random(B).astype(np.float32)
    for f in [(None, None, None), (k, None, None), (None, p, None), (None, None, m), (k, p, m)]:
        idx, lp = draw(x, T, u, *f)
        check_rows(h, T, u, *f, idx, lp)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sd", [0.0, 1e-3, 0.3, 12.0])
def test_flat_and_peaked_rows(dtype, sd):
    """Thousands of ties, tens of thousands of kept elements, one-token sets."""
    rng = np.random.default_rng(17)
    B, V = 24, 20011
    x, h = logits(rng, B, V, dtype, sd=sd)
    T = rng.uniform(0.7, 1.5, B).astype(np.float32)
    k = rng.integers(1, V, B).astype(np.int32)
    p = rng.uniform(0.3, 0.99, B).astype(np.float32)
    m = rng.uniform(0.5, 1.0, B).astype(np.float32)
    u = rng.random(B).astype(np.float32)
    u[:3] = [0.0, 1 - 2.0 ** -24, 0.5]
    for f in [(None, None, None), (k, None, None), (None, p, None), (k, p, None), (k, p, m)]:
        idx, lp = draw(x, T, u, *f)
        check_rows(h, T, u, *f, idx, lp)


def test_ties_go_to_the_lowest_index():
    x = torch.zeros(6, 1000, device="cuda")
    x[:, 500] = 1.0
    u = np.float32([0.0, 0.999, 0.999, 0.999, 0.999, 0.999])
    k = np.int32([1, 1, 2, 3, 501, 502])
    idx, lp = draw(x, np.ones(6, np.float32), u, k=k)
    assert idx.tolist() == [500, 500, 500, 500, 500, 501]
    check_rows(x.cpu().numpy(), np.ones(6), u, k, None, None, idx, lp)
    # -0 and +0 are one value
    x[:, 0::2] *= -1.0
    x[:, 500] = 1.0
    idx, _ = draw(x, np.ones(6, np.float32), np.full(6, 0.2, np.float32), k=np.full(6, 3, np.int32))
    check_rows(x.cpu().numpy(), np.ones(6), np.full(6, 0.2), np.full(6, 3), None, None, idx, None)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [3, 77, 5000])
def test_special_values(dtype, V):
    rng = np.random.default_rng(V)
    x, _ = logits(rng, 8, V, dtype)
    big = torch.finfo(TYPES[dtype]).max
    x[0] = -math.inf
    x[1] = math.nan
    x[2, 1:] = -math.inf
    x[3, V // 2:] = math.inf
    x[4, ::2] = math.nan
    x[5] = -big
    x[6, :] = -math.inf
    x[6, V - 1] = -big
    x[7, 0] = big
    h = x.float().cpu().numpy()
    u = np.full(8, 0.7, np.float32)
    for T in (1.0, 0.0, 1e-30, 1e30, math.inf):
        Ts = np.full(8, T, np.float32)
        for f in [(None, None, None), (np.full(8, 2, np.int32), np.full(8, 0.9, np.float32),
                                       np.full(8, 0.1, np.float32))]:
            idx, lp = draw(x, Ts, u, *f)
            ref = [du.draw(h[b], T, u[b], *[0 if f[0] is None else f[0][b],
                                            1.0 if f[1] is None else f[1][b],
                                            0.0 if f[2] is None else f[2][b]]) for b in range(8)]
            assert idx.tolist() == [r[0] for r in ref], (T, f[0] is None)
            assert np.allclose(lp, [r[1] for r in ref], rtol=2.0 ** -23, atol=1e-9)
            assert idx[0] == -1 and idx[1] == -1 and lp[0] == -math.inf


def test_uniform_outside_the_interval():
    x = torch.zeros(6, 64, device="cuda")
    u = np.float32([-1, np.nan, 1.0, 2.0, np.inf, -np.inf])
    idx, _ = draw(x, np.ones(6, np.float32), u)
    assert idx.tolist() == [0, 0, 63, 63, 63, 0]


def test_extreme_temperatures_and_magnitudes():
    rng = np.random.default_rng(3)
    x, h = logits(rng, 12, 3001, "f32")
    for scale, T in [(1e30, 1e30), (1e-30, 1e-30), (1.0, 1e-3), (100.0, 1.0), (1e4, 30.0), (1e-38, 1e-38)]:
        xs = (x * scale).contiguous()
        hs = xs.cpu().numpy()
        Ts = np.full(12, T, np.float32)
        u = rng.random(12).astype(np.float32)
        idx, lp = draw(xs, Ts, u, p=np.full(12, 0.95, np.float32))
        check_rows(hs, Ts, u, None, np.full(12, 0.95, np.float32), None, idx, lp)


def test_many_rows_and_batch_shapes():
    """Batches from one row to several waves give each row the same draw."""
    rng = np.random.default_rng(8)
    V = 30011
    x, h = logits(rng, 700, V, "bf16", sd=2.0)
    T, k, p, m = settings(rng, 700)
    u = rng.random(700).astype(np.float32)
    idx, lp = draw(x, T, u, k, p, m)
    check_rows(h[:60], T, u, k, p, m, idx[:60], lp[:60])
    for B in (1, 2, 9, 60, 200):
        i, l = draw(x[:B], T[:B], u[:B], k[:B], p[:B], m[:B])
        assert np.array_equal(i, idx[:B]) and np.array_equal(l, lp[:B], equal_nan=True)
    assert gs.filtered_categorical(x[:0], dev(T[:0]), dev(u[:0])).numel() == 0


def test_distribution():
    """Evenly spaced uniforms hit each token as often as its probability says,
    to one draw."""
    rng = np.random.default_rng(2)
    V, N = 50, 20000
    x = torch.from_numpy(rng.standard_normal(V).astype(np.float32)).cuda().expand(N, V).contiguous()
    u = ((np.arange(N) + 0.5) / N).astype(np.float32)
    idx, _ = draw(x, np.ones(N, np.float32), u, p=np.full(N, 0.8, np.float32))
    w, _ = du.filter_set(x[0].cpu().numpy(), 1.0, p=0.8)
    assert (np.abs(np.bincount(idx, minlength=V) - N * w / w.sum()) <= 1.5).all()


def test_scalars_streams_and_graphs():
    rng = np.random.default_rng(4)
    x, h = logits(rng, 10, 5003, "f16")
    u = rng.random(10).astype(np.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        idx = gs.filtered_categorical(x, 0.8, dev(u), top_k=40, top_p=0.9, min_p=0.01)
    side.synchronize()
    f = (np.full(10, 40), np.full(10, 0.9), np.full(10, 0.01))
    check_rows(h, np.full(10, 0.8), u, *f, idx.cpu().numpy(), None)
    T, U = torch.full((10,), 0.8, device="cuda"), dev(u)
    out, lp = torch.zeros(10, dtype=torch.int64, device="cuda"), torch.zeros(10, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gs.filtered_categorical(x, T, U, out=out, logprob=lp)
        gs.filtered_categorical(x, T, U, out=out, logprob=lp)
    for _ in range(3):
        U.copy_(torch.rand(10, device="cuda"))
        g.replay()
        check_rows(h, np.full(10, 0.8), U.cpu().numpy(), None, None, None, out.cpu().numpy(),
                   lp.cpu().numpy())


def test_draw_from_constrained_logits():
    """Logits written by process_logits just before are what is drawn from."""
    x = torch.randn(40, 4096, device="cuda")
    mask = torch.randint(-2 ** 31, 2 ** 31 - 1, (40, 128), device="cuda").int()
    u = torch.rand(40, device="cuda")
    y = torch.empty_like(x)
    for _ in range(5):
        x.normal_()
        gs.process_logits(x, mask=mask, out=y)
        idx = gs.filtered_categorical(y, 1.0, u, top_p=0.9)
        check_rows(y.cpu().numpy(), np.ones(40), u.cpu().numpy(), None, np.full(40, 0.9), None,
                   idx.cpu().numpy(), None)


def test_refusals_of_the_binding():
    x = torch.zeros(3, 8, device="cuda")
    u = torch.rand(3, device="cuda")
    for kw in (dict(uniform=u[:2]), dict(uniform=u.double()), dict(top_k=u), dict(top_p=u[:1]),
               dict(min_p=u.cpu()), dict(logprob=u.double()), dict(out=u)):
        with pytest.raises((ValueError, TypeError)):
            gs.filtered_categorical(x, 1.0, **{"uniform": u, **kw})
    with pytest.raises(ValueError):
        gs.filtered_categorical(x.t(), 1.0, u)


# ---- verification ---------------------------------------------------------------
def request_rows(rng, n, most, empty=0.1):
    lengths = rng.integers(1, most + 2, n)
    lengths[rng.random(n) < empty] = 0
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)


def run_verify(x, draft, offsets, T, u, d, q=None, k=None, p=None, m=None, **kw):
    out = torch.full((x.shape[0],), -2, dtype=torch.int64, device="cuda")
    out, count = gs.verify_drafts(x, dev(draft), dev(offsets), dev(T), dev(u), dev(d), probs=q,
                                  top_k=dev(k), top_p=dev(p), min_p=dev(m), out=out, **kw)
    return out.cpu().numpy(), count.cpu().numpy()


def check_verify(h, draft, offsets, T, u, d, q, k, p, m, out, count):
    ref, rc, gaps = du.verify(h, draft, offsets, T, u, d, q, k, p, m)
    tol = du.tolerance(h.shape[1])
    near = 0
    for i in range(len(offsets) - 1):
        rows = slice(max(0, offsets[i]), min(len(h), offsets[i + 1]))
        if gaps[i] <= 2 * tol:
            near += 1
            continue
        assert count[i] == rc[i] and np.array_equal(out[rows], ref[rows]), \
            (i, out[rows], ref[rows], count[i], rc[i], gaps[i])
    outside = ref == -2
    assert (out[outside] == -2).all()
    assert near <= max(1, len(offsets) // 50), near


@pytest.mark.parametrize("probs", [False, True])
@pytest.mark.parametrize("dtype,V,n,most,pitch", [
    ("f32", 1, 5, 2, 0), ("f32", 3, 30, 4, 0), ("bf16", 50, 40, 1, 3), ("f16", 1003, 20, 7, 1),
    ("f32", 4096, 12, 3, 0), ("bf16", 32768, 9, 4, 0), ("f16", 100003, 3, 2, 5)])
def test_verify(dtype, V, n, most, pitch, probs):
    rng = np.random.default_rng(V + n)
    offsets = request_rows(rng, n, most)
    R = int(offsets[-1]) + 3  # rows behind the last request
    x, h = logits(rng, R, V, dtype, pitch=pitch)
    q = None
    near = h + rng.standard_normal(h.shape) * 0.7
    if probs:
        e = np.exp(near - near.max(1, keepdims=True))
        qh = (e / e.sum(1, keepdims=True)).astype(np.float32)
        buf = torch.zeros(R, V + pitch, device="cuda")
        q = buf[:, :V]
        q.copy_(torch.from_numpy(qh))
        draft = np.array([rng.choice(V, p=r / r.sum()) for r in qh.astype(np.float64)])
    else:
        qh = None
        draft = near.argmax(1)
    draft = draft.astype(np.int64)
    for f in (False, True):
        T, k, p, m = settings(rng, n)
        if not f:
            k = p = m = None
        u, d = rng.random(R).astype(np.float32), rng.random(n).astype(np.float32)
        out, count = run_verify(x, draft, offsets, T, u, d, q, k, p, m)
        check_verify(h, draft, offsets, T, u, d, qh, k, p, m, out, count)


def test_verify_special_requests():
    """No rows, rows without candidates, drafts outside the vocabulary, greedy
    requests, +inf rows, all accepted, none accepted."""
    rng = np.random.default_rng(1)
    V = 500
    offsets = np.array([0, 0, 3, 5, 7, 9, 12, 14, 14], np.int64)
    x, h = logits(rng, 14, V, "f32")
    x[3] = -math.inf
    x[5, 100:200] = math.inf
    h = x.cpu().numpy()
    best = h.argmax(1)
    draft = best.copy()
    draft[7] = -1
    draft[9] = V
    T = np.float32([1, 1, 1, 1, 0.5, 0, 1, 1])
    u = np.full(14, 1e-6, np.float32)
    d = rng.random(8).astype(np.float32)
    for q in (None, np.full((14, V), 1.0 / V, np.float32)):
        for k in (None, np.full(8, 3, np.int32)):
            qd = None if q is None else dev(q)
            out, count = run_verify(x, draft, offsets, T, u, d, qd, k)
            check_verify(h, draft, offsets, T, u, d, q, k, None, None, out, count)
            assert count[0] == 0 and count[7] == 0 and out[3] == -1 and count[2] == 0


def test_verify_probabilities_equal_to_the_targets():
    """p - q is nothing but rounding where q is p: the draft is accepted for
    every u; where q is above p everywhere the draw is from p."""
    rng = np.random.default_rng(6)
    x, h = logits(rng, 8, 700, "f32")
    e = np.exp(h.astype(np.float64))
    q = (e / e.sum(1, keepdims=True)).astype(np.float32)
    draft = h.argmax(1).astype(np.int64)
    offsets = np.arange(0, 9, 2).astype(np.int64)
    u, d = np.full(8, 0.999, np.float32), rng.random(4).astype(np.float32)
    out, count = run_verify(x, draft, offsets, np.ones(4, np.float32), u, d, dev(q))
    assert count.tolist() == [2] * 4 and np.array_equal(out[::2], draft[::2])
    big = np.ones_like(q)
    out, count = run_verify(x, draft, offsets, np.ones(4, np.float32), u, d, dev(big))
    check_verify(h, draft, offsets, np.ones(4), u, d, big, None, None, None, out, count)
    assert count.tolist() == [1] * 4
    bad = q.copy()
    bad[:, ::3] = np.nan
    bad[:, 1::3] *= -1
    out, count = run_verify(x, draft, offsets, np.ones(4, np.float32), u, d, dev(bad))
    check_verify(h, draft, offsets, np.ones(4), u, d, bad, None, None, None, out, count)


def test_verify_distribution():
    """Whatever the drafts, the first token's distribution is the target's."""
    rng = np.random.default_rng(9)
    V, N = 12, 60000
    h = rng.standard_normal((2, V)).astype(np.float32)
    q = np.exp(rng.standard_normal(V))
    q = (q / q.sum()).astype(np.float32)
    x = torch.from_numpy(np.tile(h, (N, 1))).cuda()
    draft = rng.choice(V, size=2 * N, p=q.astype(np.float64) / q.sum(dtype=np.float64)).astype(np.int64)
    out, _ = run_verify(x, draft, 2 * np.arange(N + 1), np.ones(N, np.float32),
                        rng.random(2 * N).astype(np.float32), rng.random(N).astype(np.float32),
                        dev(np.tile(q, (2 * N, 1))))
    w = np.exp(h[0].astype(np.float64))
    w /= w.sum()
    seen = np.bincount(out[::2], minlength=V)
    chi = ((seen - N * w) ** 2 / (N * w)).sum()
    assert chi < 40, chi  # 11 degrees of freedom: p < 4e-5


def test_verify_malformed_offsets_stay_inside():
    rng = np.random.default_rng(12)
    x, _ = logits(rng, 6, 100, "f32")
    guard = torch.full((10,), -7, dtype=torch.int64, device="cuda")
    for offsets in ([-5, 3, 100], [4, 2, 6], [2, 2, 2], [6, 9, 12], [0, 1 << 40, -(1 << 40)]):
        guard.fill_(-7)
        count = torch.zeros(2, dtype=torch.int32, device="cuda")
        gs.verify_drafts(x, torch.zeros(6, dtype=torch.int64, device="cuda"), dev(np.int64(offsets)),
                         1.0, 0.5, 0.5, out=guard[2:8], count=count)
        assert (guard[:2] == -7).all() and (guard[8:] == -7).all()
        assert bool((count >= 0).all()) and bool((count <= 6).all())


def test_verify_in_a_graph_and_workspaces():
    rng = np.random.default_rng(13)
    offsets = np.array([0, 3, 4, 8], np.int64)
    x, h = logits(rng, 8, 2000, "bf16")
    draft = h.argmax(1).astype(np.int64)
    T = np.ones(3, np.float32)
    u, d = torch.rand(8, device="cuda"), torch.rand(3, device="cuda")
    ws = gs.new_verify_workspace(8)
    ws.fill_(255)
    out = torch.zeros(8, dtype=torch.int64, device="cuda")
    count = torch.zeros(3, dtype=torch.int32, device="cuda")
    D, O, Td = dev(draft), dev(offsets), dev(T)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gs.verify_drafts(x, D, O, Td, u, d, out=out, count=count, workspace=ws)
    for _ in range(3):
        u.uniform_()
        d.uniform_()
        g.replay()
        check_verify(h, draft, offsets, T, u.cpu().numpy(), d.cpu().numpy(), None, None, None, None,
                     out.cpu().numpy(), count.cpu().numpy())
    with pytest.raises(ValueError):
        gs.verify_drafts(x, D, O, Td, u, d, workspace=ws[:64])
    with pytest.raises(ValueError):
        gs.verify_drafts(x, D, O, Td, u, d, probs=torch.zeros(8, 1999, device="cuda"))


# ---- long rows, several streams, many requests ------------------------------------
@pytest.mark.parametrize("dtype,V,B", [("f32", 6000011, 1), ("bf16", 524309, 3)])
def test_long_rows(dtype, V, B):
    """Vocabularies past 2^18 take powers of two off their weights; past the shared
    memory for the units' maxima no list is made."""
    rng = np.random.default_rng(V)
    x, h = logits(rng, B, V, dtype)
    T, u = np.full(B, 0.9, np.float32), rng.random(B).astype(np.float32)
    for f in [(None, None, None), (np.full(B, 40, np.int32), None, None),
              (None, np.full(B, 0.7, np.float32), None), (None, None, np.full(B, 0.2, np.float32))]:
        idx, lp = draw(x, T, u, *f)
        # a unit of the weights is 2^-44 of the largest one times the powers taken off
        tol = 2.0 ** -38 + V * 2.0 ** -44 * max(1, 2.0 ** math.ceil(math.log2(V) - 18))
        check_rows(h, T, u, *f, idx, lp, tol=tol)


@pytest.mark.parametrize("B", [305, 333, 1200])
def test_batches_past_one_wave_with_long_sets_among_them(B):
    rng = np.random.default_rng(B)
    V = 16384
    x, h = logits(rng, B, V, "bf16", sd=2.5)
    T = rng.uniform(0.6, 1.2, B).astype(np.float32)
    T[::37] = 8.0  # nuclei of thousands
    p = np.full(B, 0.95, np.float32)
    k = np.where(np.arange(B) % 5 == 0, 3000, 0).astype(np.int32)
    u = rng.random(B).astype(np.float32)
    idx, lp = draw(x, T, u, k, p)
    some = np.unique(np.concatenate([np.arange(0, B, 37), np.arange(0, B, 25), [B - 1]]))
    check_rows(h[some], T[some], u[some], k[some], p[some], None, idx[some], lp[some])


def test_equal_logits_at_the_end_of_long_sets():
    """More equal logits than a list holds, in rows that differ elsewhere."""
    rng = np.random.default_rng(31)
    B, V = 6, 40000
    x = torch.from_numpy(rng.integers(0, 6, (B, V)).astype(np.float32)).cuda()
    h = x.cpu().numpy()
    u = rng.random(B).astype(np.float32)
    for T in (0.3, 1.0, 5.0):
        for f in [(np.full(B, 9000, np.int32), None, None), (None, np.full(B, 0.6, np.float32), None),
                  (np.full(B, 20000, np.int32), np.full(B, 0.9, np.float32), np.full(B, 1e-3, np.float32))]:
            idx, lp = draw(x, np.full(B, T, np.float32), u, *f)
            check_rows(h, np.full(B, T), u, *f, idx, lp)


def test_two_streams_at_once():
    rng = np.random.default_rng(77)
    x, h = logits(rng, 400, 20000, "bf16", sd=2.5)
    T, u = np.full(400, 0.9, np.float32), rng.random(400).astype(np.float32)
    Td, U = dev(T), dev(u)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    torch.cuda.synchronize()
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(gs.filtered_categorical(x, Td, U, top_p=0.9))
    torch.cuda.synchronize()
    assert all(torch.equal(o, outs[0]) for o in outs)
    some = np.arange(0, 400, 20)
    check_rows(h[some], T[some], u[some], None, np.full(20, 0.9), None, outs[0].cpu().numpy()[some], None)


def test_verify_many_requests():
    """More rows than run at once, with filters and without, drafts of all kinds."""
    rng = np.random.default_rng(41)
    n, V = 130, 9000
    offsets = request_rows(rng, n, 5)
    R = int(offsets[-1])
    x, h = logits(rng, R, V, "bf16", sd=2.5)
    draft = np.where(rng.random(R) < 0.6, h.argmax(1), rng.integers(-1, V + 1, R)).astype(np.int64)
    e = np.exp(h + rng.standard_normal(h.shape).astype(np.float32) * 0.5)
    q = (e / e.sum(1, keepdims=True)).astype(np.float32)
    T, k, p, m = settings(rng, n)
    u, d = rng.random(R).astype(np.float32), rng.random(n).astype(np.float32)
    for qd, qh in ((None, None), (dev(q), q)):
        for f in ((None, None, None), (k, p, m)):
            out, count = run_verify(x, draft, offsets, T, u, d, qd, *f)
            check_verify(h, draft, offsets, T, u, d, qh, *f, out, count)


def test_outliers_far_above_their_warps_first_logits():
    """Rows whose maximum lies many powers of two above what a warp reads first."""
    rng = np.random.default_rng(55)
    B, V = 40, 30000
    x, h = logits(rng, B, V, "f32", sd=1.0)
    x[:, 29990:29996] += torch.linspace(20, 45, B, device="cuda")[:, None]
    x[::4, :] *= 0.2
    h = x.cpu().numpy()
    u = rng.random(B).astype(np.float32)
    for T in (0.2, 0.6, 1.0):
        for f in [(None, None, None), (None, np.full(B, 0.97, np.float32), None),
                  (np.full(B, 30, np.int32), None, None)]:
            idx, lp = draw(x, np.full(B, T, np.float32), u, *f)
            check_rows(h, np.full(B, T), u, *f, idx, lp)


def test_verify_of_one_token_sets_and_no_rows():
    """Greedy rows take their draft unless u q is 1 or more; a call without rows."""
    x = torch.zeros(4, 50, device="cuda")
    x[:, 7] = 1.0
    offsets, draft = np.array([0, 2, 4], np.int64), np.array([7, 0, 7, 0], np.int64)
    q = np.zeros((4, 50), np.float32)
    q[0, 7], q[2, 7] = 1.0, 4.0
    u, d = np.full(4, 0.5, np.float32), np.full(2, 0.5, np.float32)
    out, count = run_verify(x, draft, offsets, np.zeros(2, np.float32), u, d, dev(q))
    assert out.tolist() == [7, 7, 7, -1] and count.tolist() == [2, 1]
    check_verify(x.cpu().numpy(), draft, offsets, np.zeros(2), u, d, q, None, None, None, out, count)
    tokens, count = gs.verify_drafts(x[:0], dev(draft[:0]), dev(np.zeros(4, np.int64)), 1.0,
                                     dev(u[:0]), torch.zeros(3, device="cuda"))
    assert tokens.numel() == 0 and count.tolist() == [0, 0, 0]
