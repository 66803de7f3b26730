"""Host-side checks of the draw from given random numbers, the verification of
drafts and the page tables (no GPU needed): bad arguments are rejected with the
documented status before the device is touched, empty calls succeed, and the
Python layer refuses unsuitable tensors. The 64-bit definitions that the GPU
tests compare with are pinned on small cases."""
import ctypes

import numpy as np
import pytest

import token_sampling_logits_gb300 as gs
from tests import draw_util as du

FAKE = 1 << 20  # 16-byte aligned fake device address; never dereferenced
BAD, OK, WS = gs.ERR_INVALID_ARG, gs.OK, gs.ERR_WORKSPACE


def call_draw(**kw):
    a = dict(logits=FAKE, dtype=gs.F32, B=2, V=10, ld=10, T=FAKE, u=FAKE, k=FAKE, p=FAKE, m=FAKE,
             out=FAKE, lp=FAKE)
    a.update(kw)
    return gs.lib().gsample_filtered_categorical(
        a["logits"], a["dtype"], a["B"], a["V"], a["ld"], a["T"], a["u"], a["k"], a["p"], a["m"],
        a["out"], a["lp"], None)


@pytest.mark.parametrize("kw", [
    dict(logits=None), dict(logits=FAKE + 2), dict(dtype=3), dict(B=-1), dict(V=0), dict(ld=9),
    dict(V=1 << 31, ld=1 << 31), dict(T=None), dict(u=None), dict(out=None), dict(T=FAKE + 2),
    dict(u=FAKE + 1), dict(k=FAKE + 2), dict(p=FAKE + 2), dict(m=FAKE + 2), dict(out=FAKE + 4),
    dict(lp=FAKE + 2), dict(B=(1 << 27) + 1), dict(ld=1 << 62)])
def test_draw_refusals(kw):
    assert call_draw(**kw) == BAD


def test_empty_draw():
    assert call_draw(B=0, logits=None, T=None, u=None, out=None) == OK
    assert call_draw(B=0, V=0) == BAD


def call_verify(**kw):
    a = dict(logits=FAKE, dtype=gs.F32, R=5, V=10, ld=10, n=2, offsets=FAKE, draft=FAKE,
             probs=FAKE, pld=10, T=FAKE, k=FAKE, p=FAKE, m=FAKE, u=FAKE, d=FAKE, out=FAKE,
             count=FAKE, ws=FAKE)
    a.update(kw)
    return gs.lib().gsample_verify_drafts(
        a["logits"], a["dtype"], a["R"], a["V"], a["ld"], a["n"], a["offsets"], a["draft"],
        a["probs"], a["pld"], a["T"], a["k"], a["p"], a["m"], a["u"], a["d"], a["out"], a["count"],
        a["ws"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), BAD), (dict(logits=FAKE + 1), BAD), (dict(dtype=-1), BAD),
    (dict(R=-1), BAD), (dict(n=-1), BAD), (dict(n=1 << 27), BAD), (dict(R=1 << 27), BAD),
    (dict(offsets=None), BAD), (dict(offsets=FAKE + 4), BAD), (dict(draft=None), BAD),
    (dict(draft=FAKE + 4), BAD), (dict(probs=FAKE + 2), BAD), (dict(pld=9), BAD),
    (dict(pld=1 << 62), BAD), (dict(T=None), BAD), (dict(T=FAKE + 2), BAD), (dict(k=FAKE + 1), BAD),
    (dict(p=FAKE + 1), BAD), (dict(m=FAKE + 1), BAD), (dict(u=None), BAD), (dict(u=FAKE + 2), BAD),
    (dict(d=None), BAD), (dict(d=FAKE + 2), BAD), (dict(out=None), BAD), (dict(out=FAKE + 4), BAD),
    (dict(count=None), BAD), (dict(count=FAKE + 2), BAD), (dict(ws=None), WS),
    (dict(ws=FAKE + 8), WS), (dict(n=0), OK), (dict(n=0, R=0, logits=None, offsets=None, ws=None), OK)])
def test_verify_arguments(kw, status):
    assert call_verify(**kw) == status


def test_verify_workspace():
    f = gs.lib().gsample_verify_workspace_bytes
    assert [f(r) for r in (-1, 0, 1, 5)] == [0, 0, 32, 160]


def pages(**kw):
    a = dict(table=FAKE, length=FAKE, free=FAKE, count=FAKE, rows=8, ld=4, pages=20, page=16)
    a.update(kw)
    return gs._PagesC(a["table"], a["length"], a["free"], a["count"], a["rows"], a["ld"],
                      a["pages"], a["page"])


def call_extend(s, **kw):
    a = dict(slot=FAKE, n=3, offsets=FAKE, total=9, start=FAKE, maps=FAKE, length=FAKE,
             table=FAKE, cols=4, ld=4)
    a.update(kw)
    return gs.lib().gsample_pages_extend(
        ctypes.byref(s) if s is not None else None, a["slot"], a["n"], a["offsets"], a["total"],
        a["start"], a["maps"], a["length"], a["table"], a["cols"], a["ld"], None)


def call_trim(s, **kw):
    a = dict(slot=FAKE, n=3, start=FAKE, keep=FAKE)
    a.update(kw)
    return gs.lib().gsample_pages_trim(ctypes.byref(s) if s is not None else None, a["slot"],
                                       a["n"], a["start"], a["keep"], None)


@pytest.mark.parametrize("kw", [
    dict(table=None), dict(length=None), dict(free=None), dict(count=None), dict(table=FAKE + 2),
    dict(length=FAKE + 1), dict(free=FAKE + 2), dict(count=FAKE + 3), dict(rows=0),
    dict(rows=65537), dict(ld=0), dict(pages=0), dict(pages=1 << 31), dict(page=0), dict(page=-4),
    dict(ld=1 << 27, page=16)])
def test_bad_page_states_are_refused(kw):
    assert call_extend(pages(**kw)) == BAD
    assert call_trim(pages(**kw)) == BAD
    assert call_extend(pages(**kw), n=0) == BAD


def test_a_null_page_state_is_refused():
    assert call_extend(None) == BAD and call_trim(None) == BAD


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), BAD), (dict(n=1 << 31), BAD), (dict(total=-1), BAD), (dict(total=1 << 31), BAD),
    (dict(offsets=None), BAD), (dict(slot=None, n=9), BAD), (dict(start=None), BAD),
    (dict(maps=None), BAD), (dict(slot=FAKE + 2), BAD), (dict(offsets=FAKE + 4), BAD),
    (dict(start=FAKE + 2), BAD), (dict(maps=FAKE + 4), BAD), (dict(length=FAKE + 1), BAD),
    (dict(table=FAKE + 1), BAD), (dict(cols=-1), BAD), (dict(cols=5), BAD), (dict(ld=1 << 62), BAD),
    (dict(n=0), OK), (dict(n=0, start=None, maps=None, slot=None), OK)])
def test_extend_arguments(kw, status):
    assert call_extend(pages(), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), BAD), (dict(n=1 << 31), BAD), (dict(slot=None, n=9), BAD),
    (dict(slot=FAKE + 1), BAD), (dict(start=FAKE + 2), BAD), (dict(keep=FAKE + 2), BAD),
    (dict(n=0), OK)])
def test_trim_arguments(kw, status):
    assert call_trim(pages(), **kw) == status


def test_debug_weights_arguments():
    f = gs.lib().gsample_debug_weights
    assert f(FAKE, 4, 1.0, 0.0, FAKE, None) == BAD
    assert f(FAKE, 4, float("inf"), 1.0, FAKE, None) == BAD
    assert f(None, 4, 1.0, 1.0, FAKE, None) == BAD
    assert f(FAKE, 4, 1.0, 1.0, FAKE + 4, None) == BAD
    assert f(None, 0, 1.0, 1.0, None, None) == OK


def test_the_python_layer_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        gs.filtered_categorical(x, 1.0, 0.5)
    with pytest.raises(ValueError):
        gs.verify_drafts(x, torch.zeros(2).long(), torch.tensor([0, 2]), 1.0, 0.5, 0.5)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        gs.PageState(i.view(2, 2), i[:2], i, i[:1], 16)


def test_the_kernels_wait_before_they_may_exit():
    """As every kernel of the library (tests/test_launch_order.py), those of the
    shared header: the first wait comes before the first return."""
    import os
    import re

    from token_sampling_logits_gb300 import build

    text = open(os.path.join(build.CSRC, "gsample_draw.cuh")).read()
    text = re.sub(r"//[^\n]*", " ", text)
    found = 0
    for m in re.finditer(r"__global__ void __launch_bounds__\([^)]*\)\s*(\w+)\(", text):
        body = text[text.index("{", m.end()):]
        wait, leave = body.index("pdl_wait_then_release()"), body.index("return;")
        assert wait < leave, m.group(1)
        assert "__ldcg" not in body[:wait] and "__ldg" not in body[:wait]
        found += 1
    assert found == 2


# ---- the definitions ------------------------------------------------------------
def test_the_filter_set_of_a_small_row():
    x = np.log([0.4, 0.1, 0.3, 0.1, 0.1]).astype(np.float32)
    some = lambda **kw: np.flatnonzero(du.filter_set(x, 1.0, **kw)[0]).tolist()  # noqa: E731
    assert some() == [0, 1, 2, 3, 4]
    assert some(k=2) == [0, 2] and some(k=3) == [0, 1, 2] and some(k=99) == [0, 1, 2, 3, 4]
    assert some(p=0.5) == [0, 2] and some(p=0.75) == [0, 1, 2] and some(p=0.0) == [0]
    assert some(p=float("nan")) == [0, 1, 2, 3, 4]
    assert some(m=0.5) == [0, 2] and some(m=1.0) == [0] and some(m=7.0) == [0]
    assert some(k=4, p=0.75, m=0.9) == [0]


def test_the_draw_of_a_small_row():
    x = np.log([0.25, 0.25, 0.5]).astype(np.float32)
    assert [du.draw(x, 1.0, u)[0] for u in (0.0, 0.2, 0.3, 0.49, 0.51, 1.5, -1)] == [0, 0, 1, 1, 2, 2, 0]
    assert du.draw(x, 0.0, 0.0)[0] == 2 and du.draw(x * np.nan, 1.0, 0.5)[0] == -1


def test_verification_of_a_small_request():
    x = np.log(np.array([[0.5, 0.25, 0.25], [0.5, 0.25, 0.25], [0.1, 0.1, 0.8]])).astype(np.float32)
    q = np.array([[1.0, 0, 0], [0, 1.0, 0], [0, 0, 0]])
    run = lambda u, d: du.verify(x, [0, 1, 0], [0, 3], [1.0], u, [d], q)  # noqa: E731
    out, count, _ = run([0.4, 0.2, 0], 0.5)
    assert out.tolist() == [0, 1, 2] and count[0] == 3
    out, count, _ = run([0.4, 0.3, 0], 0.5)  # rest (0.5, 0, 0.25)
    assert out.tolist() == [0, 0, -1] and count[0] == 2
    out, count, _ = run([0.6, 0.3, 0], 0.4)  # rest (0, 0.25, 0.25)
    assert out.tolist() == [1, -1, -1] and count[0] == 1


def test_pages_of_a_plain_scheduler():
    s = du.Pages(3, 6, 4, 3)
    assert s.extend([5, 4], [1, 0]) == ([0, 0], [[0, 1, 2, 3, 4], [8, 9, 10, 11]], [5, 4], [[0, 1], [2]])
    assert s.extend([9, 1, 1], [2, 1, 0])[0] == [0, 5, -1]  # no page left for the last
    s.trim([2, 1], [0, 5], [0, 0])
    assert s.free == [5, 4, 3] and s.length == [4, 5, 0]
