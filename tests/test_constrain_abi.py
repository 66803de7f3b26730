"""Host-side checks of the logit-constraint entry points (no GPU needed): bad
arguments are rejected with the documented status before the device is
touched, empty calls succeed, and the Python layer refuses unsuitable tensors."""
import ctypes

import numpy as np
import pytest

import token_sampling_logits_gb300 as gs
from tests import constrain_util as cu

FAKE = 1 << 20  # 16-byte aligned fake device address; never dereferenced
BAD, OK = gs.ERR_INVALID_ARG, gs.OK


def state(**kw):
    a = dict(history=FAKE, bias=FAKE, touched=FAKE, rows=8, vocab=100, ld=128)
    a.update(kw)
    return gs._StateC(a["history"], a["bias"], a["touched"], a["rows"], a["vocab"], a["ld"])


def ref(s):
    return ctypes.byref(s) if s is not None else None


BAD_STATES = [dict(history=None), dict(touched=None), dict(history=FAKE + 4), dict(bias=FAKE + 8),
              dict(touched=FAKE + 2), dict(rows=0), dict(rows=-1), dict(vocab=0),
              dict(vocab=1 << 31, ld=1 << 31), dict(ld=96), dict(ld=120), dict(ld=0),
              dict(rows=1 << 60)]


def test_state_ld():
    ld = gs.lib().gsample_logit_state_ld
    assert [ld(v) for v in (1, 31, 32, 33, 151936)] == [32, 32, 32, 64, 151936]
    assert ld(0) == 0 and ld(-5) == 0


@pytest.mark.parametrize("kw", BAD_STATES)
def test_bad_states_are_refused_by_every_call(kw):
    L, s = gs.lib(), state(**kw)
    assert L.gsample_state_reset(ref(s), None, 0, None) == BAD
    assert L.gsample_history_append(ref(s), None, 0, FAKE, 0, FAKE, 0, None) == BAD
    assert L.gsample_bias_set(ref(s), None, 0, FAKE, FAKE, 0, FAKE, None) == BAD
    c = gs._ConstraintsC()
    c.state, c.keep = ctypes.addressof(s), s
    c.slot = FAKE
    V = s.vocab if 0 < s.vocab < (1 << 31) - 128 else 100
    assert L.gsample_process_logits(FAKE, gs.F32, 2, V, V, ctypes.byref(c), FAKE + (1 << 30),
                                    gs.F32, V, None) == BAD
    assert L.gsample_constrained_gumbel_argmax(FAKE, gs.F32, 2, V, V, FAKE, FAKE, FAKE,
                                               ctypes.byref(c), FAKE, FAKE, None) == BAD


def test_a_null_state_is_refused():
    L = gs.lib()
    assert L.gsample_state_reset(None, None, 0, None) == BAD
    assert L.gsample_history_append(None, None, 0, FAKE, 0, FAKE, 0, None) == BAD
    assert L.gsample_bias_set(None, None, 0, FAKE, FAKE, 0, FAKE, None) == BAD


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), BAD),
    (dict(n=1 << 31), BAD),
    (dict(total=-1), BAD),
    (dict(total=5), BAD),  # no offsets: one token a request
    (dict(slot=None, n=9, total=9), BAD),  # more requests than state rows
    (dict(slot=FAKE + 2), BAD),
    (dict(tokens=None), BAD),
    (dict(tokens=FAKE + 4), BAD),
    (dict(offsets=FAKE + 4), BAD),
    (dict(values=FAKE + 2), BAD),
    (dict(values=None), BAD),
    (dict(n=0, total=0), OK),
    (dict(n=0, total=0, tokens=None, slot=None, values=None), OK),
    (dict(total=0, offsets=FAKE, tokens=None), OK),
])
def test_list_arguments(kw, status):
    a = dict(slot=FAKE, n=4, tokens=FAKE, values=FAKE, total=4, offsets=None)
    a.update(kw)
    L, s = gs.lib(), state()
    got = L.gsample_bias_set(ref(s), a["slot"], a["n"], a["tokens"], a["values"], a["total"],
                             a["offsets"], None)
    assert got == status
    if "values" not in kw:
        for kind in (0, 1):
            assert L.gsample_history_append(ref(s), a["slot"], a["n"], a["tokens"], a["total"],
                                            a["offsets"], kind, None) == status


def test_kind_slots_and_missing_biases():
    L, s = gs.lib(), state()
    for kind in (-1, 2):
        assert L.gsample_history_append(ref(s), FAKE, 4, FAKE, 4, None, kind, None) == BAD
    assert L.gsample_state_reset(ref(s), None, 9, None) == BAD
    assert L.gsample_state_reset(ref(s), FAKE + 1, 4, None) == BAD
    assert L.gsample_state_reset(ref(s), None, 0, None) == OK
    assert L.gsample_bias_set(ref(state(bias=None)), FAKE, 4, FAKE, FAKE, 4, None, None) == BAD


def constraints(s=None, **kw):
    c = gs._ConstraintsC()
    if s is not None:
        c.state, c.keep = ctypes.addressof(s), s
    for k, v in kw.items():
        setattr(c, k, v)
    return c


CON = [
    (lambda: constraints(state(vocab=101)), BAD),  # another vocabulary
    (lambda: constraints(state(rows=3)), BAD),  # no slots: a state row for each batch row
    (lambda: constraints(state(rows=3), slot=FAKE), None),
    (lambda: constraints(state(), slot=FAKE + 2), BAD),
    (lambda: constraints(state(), repetition=FAKE + 1), BAD),
    (lambda: constraints(state(), frequency=FAKE + 2), BAD),
    (lambda: constraints(state(), presence=FAKE + 3), BAD),
    (lambda: constraints(mask=FAKE, mask_rows=4, mask_ld=3), BAD),  # 100 tokens need 4 words
    (lambda: constraints(mask=FAKE, mask_rows=3, mask_ld=4), BAD),  # no mask_row: a mask a row
    (lambda: constraints(mask=FAKE, mask_rows=-1, mask_ld=4, mask_row=FAKE), BAD),
    (lambda: constraints(mask=FAKE + 2, mask_rows=4, mask_ld=4), BAD),
    (lambda: constraints(mask=FAKE, mask_rows=4, mask_ld=4, mask_row=FAKE + 2), BAD),
    (lambda: constraints(mask=FAKE, mask_rows=1 << 40, mask_ld=1 << 40, mask_row=FAKE), BAD),
    (lambda: constraints(mask=FAKE, mask_rows=0, mask_ld=(1 << 63) - 1, mask_row=FAKE), BAD),
]


@pytest.mark.parametrize("make,status", CON)
def test_constraint_arguments(make, status):
    """B = 4, V = 100; a valid set reaches the device query, which fails here
    (or, with a GPU, is not made: B = 0)."""
    L, c = gs.lib(), make()
    far = FAKE + (1 << 30)
    for B in ((4,) if status == BAD else (0,)):
        want = OK if status is None else status
        assert L.gsample_process_logits(FAKE, gs.BF16, B, 100, 100, ctypes.byref(c), far, gs.F32,
                                        100, None) == want
        assert L.gsample_constrained_gumbel_argmax(FAKE, gs.BF16, B, 100, 100, FAKE, FAKE, FAKE,
                                                   ctypes.byref(c), FAKE, FAKE, None) == want


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), BAD), (dict(out=None), BAD), (dict(dtype=7), BAD), (dict(B=-1), BAD),
    (dict(V=0), BAD), (dict(V=1 << 31, ld=1 << 31, out_ld=1 << 31), BAD), (dict(ld=99), BAD),
    (dict(out_ld=99), BAD), (dict(logits=FAKE + 1), BAD), (dict(out=FAKE + 1), BAD),
    (dict(out_dtype=gs.F16), BAD),  # bf16 logits to f16
    (dict(dtype=gs.F32, out_dtype=gs.BF16), BAD),
    (dict(B=0), OK), (dict(B=0, logits=None, out=None), OK),
])
def test_process_arguments(kw, status):
    a = dict(logits=FAKE, dtype=gs.BF16, B=4, V=100, ld=100, out=FAKE + (1 << 30),
             out_dtype=gs.BF16, out_ld=100)
    a.update(kw)
    assert gs.lib().gsample_process_logits(a["logits"], a["dtype"], a["B"], a["V"], a["ld"], None,
                                           a["out"], a["out_dtype"], a["out_ld"], None) == status


@pytest.mark.parametrize("shift,ld,out_ld,dtype,out_dtype", [
    (4, 100, 100, 0, 0),  # one element further
    (400, 100, 100, 0, 0),  # one row further
    (0, 100, 128, 0, 0),  # the same start with another pitch
    (0, 128, 128, 1, 0),  # wider results over the logits
    (200, 128, 128, 0, 0),  # halfway into a row
    (128 * 4 * 2 - 4, 128, 128, 0, 0),  # the end of a row in the gap, its rest in the next row
])
def test_overlapping_results_are_refused(shift, ld, out_ld, dtype, out_dtype):
    L = gs.lib()
    for at in (FAKE + shift, FAKE - shift):
        assert L.gsample_process_logits(FAKE, dtype, 4, 100, ld, None, at, out_dtype, out_ld,
                                        None) == BAD


def test_interleaved_rows_of_one_pitch_are_not_an_overlap():
    """Results in the other half of each row: the call gets past its checks.
    Made only where that ends at the device query: the addresses are not real."""
    if _has_gpu():
        pytest.skip("a GPU is present")
    L = gs.lib()
    for at in (FAKE + 512, FAKE - 512, FAKE + 400, FAKE + 624):
        assert L.gsample_process_logits(FAKE, 0, 4, 100, 256, None, at, 0, 256,
                                        None) == gs.ERR_CUDA


def _has_gpu():
    torch = pytest.importorskip("torch")
    return torch.cuda.is_available()


def test_no_device_is_an_error_not_a_fallback():
    if _has_gpu():
        pytest.skip("a GPU is present")
    L, s = gs.lib(), state()
    assert L.gsample_state_reset(ref(s), FAKE, 4, None) == gs.ERR_CUDA
    assert L.gsample_history_append(ref(s), FAKE, 4, FAKE, 4, None, 1, None) == gs.ERR_CUDA
    assert L.gsample_bias_set(ref(s), FAKE, 4, FAKE, FAKE, 4, None, None) == gs.ERR_CUDA
    assert L.gsample_process_logits(FAKE, 0, 4, 100, 100, None, FAKE + (1 << 30), 0, 100,
                                    None) == gs.ERR_CUDA
    assert L.gsample_process_logits(FAKE, 0, 4, 100, 100, None, FAKE, 0, 100, None) == gs.ERR_CUDA
    assert L.gsample_constrained_gumbel_argmax(FAKE, 0, 4, 100, 100, FAKE, FAKE, FAKE, None, FAKE,
                                               FAKE, None) == gs.ERR_CUDA


@pytest.mark.parametrize("kw,status", [
    (dict(T=None), BAD), (dict(seed=None), BAD), (dict(off=None), BAD), (dict(out=None), BAD),
    (dict(ws=None), BAD), (dict(out=FAKE + 4), BAD), (dict(ws=FAKE + 8), gs.ERR_WORKSPACE),
    (dict(logits=None), BAD), (dict(V=0), BAD), (dict(ld=99), BAD), (dict(B=-1), BAD),
    (dict(B=0), OK), (dict(B=0, logits=None, out=None, ws=None, T=None), OK),
])
def test_draw_arguments(kw, status):
    a = dict(logits=FAKE, B=4, V=100, ld=100, T=FAKE, seed=FAKE, off=FAKE, out=FAKE, ws=FAKE)
    a.update(kw)
    assert gs.lib().gsample_constrained_gumbel_argmax(
        a["logits"], gs.F32, a["B"], a["V"], a["ld"], a["T"], a["seed"], a["off"], None, a["out"],
        a["ws"], None) == status


def test_python_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    z = torch.zeros(2, 32, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        gs.LogitState(z, None, z[:, :1], 32)
    with pytest.raises(ValueError, match="CUDA"):
        gs.process_logits(torch.zeros(2, 32))
    with pytest.raises(ValueError, match="CUDA"):
        gs.constrained_gumbel_argmax(torch.zeros(2, 32), 1.0, 0, 0)


# ---- the tests' own plain forms ---------------------------------------------
def test_plain_form_by_hand():
    x = np.array([[2.0, -2.0, 1.0, 0.0, -np.inf, 5.0, 3.0, np.nan]])
    h = np.array([[3, 0x80000000, 0x80000001, 1, 7, 0, 0, 0]], np.uint32)
    b = np.array([[0, 0, 1.0, 0, 4.0, -np.inf, 0, 0]])
    allowed = np.array([[1, 1, 1, 1, 1, 1, 0, 0]], bool)
    y, e = cu.constrained(x, h, b, [2.0], [0.25], [0.5], allowed)
    want = [2 / 2 - 0.75 - 0.5, -4.0, 2 / 2 - 0.25 - 0.5, 0 - 0.25 - 0.5, -np.inf, -np.inf,
            -np.inf, -np.inf]
    assert np.array_equal(y[0], want)
    assert np.array_equal(cu.binary32(x, h, b, [2.0], [0.25], [0.5], allowed)[0], want)
    y, _ = cu.constrained(x, h, b, [np.nan], [np.nan], [np.nan], allowed)
    assert np.array_equal(y[0][:4], [2.0, -2.0, 2.0, 0.0])


def test_check_values_notices_a_misrounded_value():
    x = np.full((1, 4), 10.0)
    one = np.ones((1, 4), np.uint32)
    y, e = cu.constrained(x, one, np.zeros((1, 4)), [3.0], [0.1], [0.7], np.ones((1, 4), bool))
    good = cu.binary32(x, one, np.zeros((1, 4)), [3.0], [0.1], [0.7], np.ones((1, 4), bool))
    cu.check_values(good, y, e, 0)
    for wrong in (good * np.float32(1 + 2.0 ** -20), good - np.float32(0.1)):
        with pytest.raises(AssertionError):
            cu.check_values(wrong, y, e, 0)


def test_pack_bits_layout():
    m = np.zeros((1, 70), bool)
    m[0, [0, 31, 32, 69]] = True
    assert [int(w) for w in cu.pack_bits(m)[0]] == [1 | 1 << 31, 1, 1 << 5]
