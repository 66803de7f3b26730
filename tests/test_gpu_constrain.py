"""Logit constraints on the GPU (penalties, biases, grammar masks, the state
behind them and the draw): against plain 64-bit forms, and against the library's
own sampler on the written logits."""
import ctypes

import numpy as np
import pytest

import oracle
import token_sampling_logits_gb300 as gs
import workloads as W
from tests import constrain_util as cu
from tests.gpu_util import Tally, register, to_device

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

TYPES = {W.F32: torch.float32, W.BF16: torch.bfloat16, W.F16: torch.float16}


def dev(a):
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint32:
        a = a.view(np.int32)
    return torch.from_numpy(a.copy()).cuda()


def upload(s: cu.HostState, bias=True):
    return gs.LogitState(dev(s.history), dev(s.bias) if bias else None, dev(s.words()), s.vocab)


def same_state(state, s: cu.HostState):
    assert np.array_equal(state.history.cpu().numpy().view(np.uint32), s.history)
    if state.bias is not None:
        assert np.array_equal(state.bias.cpu().numpy(), s.bias)
    assert np.array_equal(state.touched.cpu().numpy().view(np.uint32), s.words())


def ragged(rng, lengths, vocab):
    offsets = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)
    return rng.integers(0, vocab, int(offsets[-1])).astype(np.int64), offsets


# ---- the state ----------------------------------------------------------------
@pytest.mark.parametrize("vocab", [1, 5, 32, 33, 1000, 50021])
@pytest.mark.parametrize("lengths", [[0], [1], [3, 0, 700, 1], [0, 0, 0], [257, 256, 255, 1, 0]])
def test_append_ragged_lists(vocab, lengths):
    rng = np.random.default_rng([vocab, len(lengths)])
    s = cu.random_state(rng, 7, vocab)
    state = upload(s)
    tokens, offsets = ragged(rng, lengths, vocab)
    slots = rng.permutation(7)[:len(lengths)].astype(np.int32)
    for prompt in (True, False):
        gs.history_append(state, dev(tokens), slots=dev(slots), offsets=dev(offsets),
                          prompt=prompt)
        for i, r in enumerate(slots):
            s.append(r, tokens[offsets[i]:offsets[i + 1]], prompt)
    same_state(state, s)


@pytest.mark.parametrize("lengths", [[40000], [140000], [0, 70000, 1, 64000]])
def test_append_long_lists(lengths):
    """Long lists of one request are counted in tables first: few frequent
    tokens, many rare ones, and ids that are none."""
    rng = np.random.default_rng(len(lengths))
    V = 50021
    s = cu.random_state(rng, 5, V)
    state = upload(s)
    offsets = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)
    n = int(offsets[-1])
    tokens = np.minimum((float(V) ** rng.random(n)).astype(np.int64) - 1, V - 1)
    tokens[rng.random(n) < 0.01] = -1
    tokens[rng.random(n) < 0.01] = V
    slots = rng.permutation(5)[:len(lengths)].astype(np.int32)
    for prompt in (False, True):
        gs.history_append(state, dev(tokens), slots=dev(slots), offsets=dev(offsets),
                          prompt=prompt)
        for i, r in enumerate(slots):
            mine = tokens[offsets[i]:offsets[i + 1]]
            mine = mine[(mine >= 0) & (mine < V)]
            if prompt:
                s.history[r, mine] |= np.uint32(0x80000000)
            else:
                np.add.at(s.history[r], mine, np.uint32(1))
            s.touched[r, mine] = True
    same_state(state, s)


def test_append_one_token_a_row():
    rng = np.random.default_rng(1)
    s = cu.random_state(rng, 70, 333)
    state = upload(s)
    for step in range(5):
        tokens = rng.integers(-1, 333, 70)
        gs.history_append(state, dev(tokens))
        for r in range(70):
            s.append(r, [tokens[r]], False)
    same_state(state, s)


def test_ids_slots_and_positions_outside_their_ranges_are_ignored():
    s = cu.random_state(np.random.default_rng(2), 4, 100)
    state = upload(s)
    tokens = np.array([-1, 100, 127, 1 << 40, -(1 << 62), 99, 0, 50, 51, 52], np.int64)
    # positions 0..1 and 9 belong to no request; request 2 is empty
    offsets = np.array([2, 6, 7, 7, 9], np.int64)
    slots = np.array([3, 4, 0, -1], np.int32)
    gs.history_append(state, dev(tokens), slots=dev(slots), offsets=dev(offsets))
    s.append(3, tokens[2:6], False)
    gs.bias_set(state, dev(tokens), dev(np.arange(10, dtype=np.float32)), slots=dev(slots),
                offsets=dev(offsets))
    s.set_bias(3, tokens[2:6], np.arange(2, 6))
    gs.state_reset(state, slots=dev(np.array([-1, 4, 1 << 30, 2], np.int32)))
    s.reset(2)
    same_state(state, s)
    # offsets past the lists, and decreasing ones: nothing outside is read
    gs.history_append(state, dev(tokens[5:8]), slots=dev(slots[:2]),
                      offsets=dev(np.array([0, 1, 1 << 40], np.int64)), prompt=True)
    s.append(3, tokens[5:6], True)  # request 1 names no state row
    gs.bias_set(state, dev(tokens[5:8]), dev(np.full(3, 2.5, np.float32)), slots=dev(slots[:1]),
                offsets=dev(np.array([-5, 1 << 40], np.int64)))
    s.set_bias(3, tokens[5:8], np.full(3, 2.5))
    gs.bias_set(state, dev(tokens[5:8]), dev(np.full(3, 9.5, np.float32)), slots=dev(slots[:1]),
                offsets=dev(np.array([2, 1], np.int64)))
    same_state(state, s)


def test_a_slot_and_a_token_named_often():
    s = cu.HostState(3, 64)
    state = upload(s)
    tokens = np.array([7] * 1000 + [8, 7, 8], np.int64)
    slots = np.array([1, 1, 1], np.int32)
    offsets = np.array([0, 500, 500, 1003], np.int64)
    gs.history_append(state, dev(tokens), slots=dev(slots), offsets=dev(offsets))
    s.append(1, tokens, False)
    same_state(state, s)
    assert state.history[1, 7].item() == 1001


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 64, 65, 300, 1500])
def test_bias_lists_the_later_value_stays(n):
    rng = np.random.default_rng(n)
    s = cu.random_state(rng, 5, 97)
    state = upload(s)
    ids = rng.integers(-2, 99, 3 * n)
    values = rng.standard_normal(3 * n).astype(np.float32)
    offsets = np.array([0, n, n, 3 * n], np.int64)
    slots = np.array([4, 0, 2], np.int32)
    gs.bias_set(state, dev(ids), dev(values), slots=dev(slots), offsets=dev(offsets))
    for i, r in enumerate(slots):
        s.set_bias(r, ids[offsets[i]:offsets[i + 1]], values[offsets[i]:offsets[i + 1]])
    same_state(state, s)


@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("vocab,ld", [(1, 32), (40, 96), (5000, 5024)])
def test_reset_leaves_other_rows(vocab, ld, bias):
    rng = np.random.default_rng(vocab)
    s = cu.random_state(rng, 6, vocab, ld=ld, biases=6 if bias else 0)
    state = upload(s, bias)
    gs.state_reset(state, slots=dev(np.array([5, 1, 1], np.int32)))
    s.reset(5), s.reset(1)
    same_state(state, s)
    gs.state_reset(state)
    for r in range(6):
        s.reset(r)
    same_state(state, s)


# ---- the constrained logits -----------------------------------------------------
def logits_for(rng, B, V, dtype, special=True):
    x = (rng.standard_normal((B, V)) * 4).astype(np.float32)
    if special:
        x[rng.random((B, V)) < 0.02] = -np.inf
        x[rng.random((B, V)) < 0.005] = np.nan
        x[rng.random((B, V)) < 0.005] = np.inf
        x[rng.random((B, V)) < 0.01] = 0.0
    return W.roundtrip(x, dtype)


class Problem:
    """A batch with everything in use: states by slot (some rows without),
    masks by row (some without), penalties."""

    def __init__(self, seed, B, V, dtype, special=True, tokens=40, state=True, mask=True,
                 pitch=0, shift=0):
        rng = np.random.default_rng([seed, B, V, dtype])
        self.B, self.V, self.dtype = B, V, dtype
        self.x = logits_for(rng, B, V, dtype, special)
        buf = torch.zeros(B * (V + pitch) + shift + 8, dtype=TYPES[dtype], device="cuda")
        self.logits = buf[shift:shift + B * (V + pitch)].view(B, V + pitch)[:, :V]
        self.logits.copy_(torch.from_numpy(self.x))
        rows = B + 2
        self.host = cu.random_state(rng, rows, V, tokens=tokens)
        self.slots = rng.permutation(rows)[:B].astype(np.int32)
        if B > 4:
            self.slots[2] = self.slots[0]  # two rows share a request's state
            self.slots[3], self.slots[4] = -1, rows
        self.rep = rng.uniform(0.5, 2.0, B).astype(np.float32)
        self.freq = rng.uniform(-0.5, 1.0, B).astype(np.float32)
        self.pres = rng.uniform(-0.5, 1.0, B).astype(np.float32)
        for j, bad in enumerate([0.0, -1.5, np.inf, np.nan]):
            if B > 8 + j:
                self.rep[8 + j] = bad
        if B > 13:
            self.freq[12], self.pres[13] = np.nan, np.nan
        self.bits = cu.random_mask(rng, B + 1, V)
        self.mask_rows = rng.permutation(B + 1)[:B].astype(np.int32)
        if B > 6:
            self.mask_rows[5], self.mask_rows[6] = -1, B + 1
        self.with_state, self.with_mask = state, mask
        self.kw = {}
        if state:
            self.kw.update(state=upload(self.host), slots=dev(self.slots),
                           repetition=dev(self.rep), frequency=dev(self.freq),
                           presence=dev(self.pres))
        if mask:
            self.kw.update(mask=dev(cu.pack_bits(self.bits)), mask_rows=dev(self.mask_rows))

    def parts(self):
        B, V = self.B, self.V
        h, b = np.zeros((B, V), np.uint32), np.zeros((B, V), np.float32)
        if self.with_state:
            ok = (self.slots >= 0) & (self.slots < self.host.rows)
            h[ok] = self.host.history[self.slots[ok], :V]
            b[ok] = self.host.bias[self.slots[ok], :V]
        allowed = np.ones((B, V), bool)
        if self.with_mask:
            ok = (self.mask_rows >= 0) & (self.mask_rows <= B)
            allowed[ok] = self.bits[self.mask_rows[ok]]
        one = np.ones(B), np.zeros(B), np.zeros(B)
        return (self.x, h, b) + ((self.rep, self.freq, self.pres) if self.with_state else one) + \
            (allowed,)

    def want(self):
        return cu.constrained(*self.parts())


SIZES = [1, 2, 7, 8, 9, 31, 32, 33, 64, 255, 1000, 1023, 2048, 4099, 33000]


def out_values(t):
    return t.float().cpu().numpy()


@pytest.mark.parametrize("V", SIZES)
@pytest.mark.parametrize("dtype", [W.F32, W.BF16, W.F16])
@pytest.mark.parametrize("odt", ["same", "f32"])
def test_process_against_64_bits(V, dtype, odt):
    for B, pitch, shift in ((1, 0, 0), (15, 0, 0), (15, (-V) % 64, 0), (15, 3, 1)):
        p = Problem(3, B, V, dtype, pitch=pitch, shift=shift)
        code = W.F32 if odt == "f32" else dtype
        got = gs.process_logits(p.logits, out_dtype=TYPES[code], **p.kw)
        assert got.dtype == TYPES[code]
        cu.check_values(out_values(got), *p.want(), code, "B %d pitch %d" % (B, pitch))


@pytest.mark.parametrize("state,mask", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
def test_process_with_parts_absent(state, mask, dtype):
    for V in (9, 1000, 5001):
        p = Problem(4, 16, V, dtype, state=state, mask=mask)
        got = gs.process_logits(p.logits, **p.kw)
        cu.check_values(out_values(got), *p.want(), dtype)


def test_process_parameters_absent_and_scalar():
    p = Problem(5, 9, 500, W.F32, mask=False)
    kw = dict(p.kw, repetition=None, frequency=0.25, presence=None)
    p.rep[:], p.freq[:], p.pres[:] = 1, 0.25, 0
    cu.check_values(out_values(gs.process_logits(p.logits, **kw)), *p.want(), W.F32)
    # without biases, without slots and mask rows: row b uses state and mask b
    p = Problem(6, 9, 500, W.F32)
    p.host.bias[:] = 0
    p.slots, p.mask_rows = np.arange(9, dtype=np.int32), np.arange(9, dtype=np.int32)
    kw = dict(p.kw, state=upload(p.host, bias=False), slots=None, mask_rows=None)
    cu.check_values(out_values(gs.process_logits(p.logits, **kw)), *p.want(), W.F32)


@pytest.mark.parametrize("V", SIZES)
@pytest.mark.parametrize("dtype", [W.F32, W.BF16, W.F16])
def test_process_in_place(V, dtype):
    for B, pitch, shift in ((15, 0, 0), (15, (-V) % 64, 0), (15, 3, 1)):
        p = Problem(7, B, V, dtype, pitch=pitch, shift=shift)
        want = gs.process_logits(p.logits, **p.kw)
        base = p.logits._base
        before = base.clone()
        got = gs.process_logits(p.logits, out=p.logits, **p.kw)
        assert got is p.logits
        a, b = got.contiguous(), want
        bits = torch.int32 if dtype == W.F32 else torch.int16
        nan = torch.isnan(a) & torch.isnan(b)
        assert bool(((a.view(bits) == b.view(bits)) | nan).all())
        # the gaps between rows and around the batch are as they were
        edge = torch.ones_like(base, dtype=torch.bool)
        torch.as_strided(edge, (B, V), (V + pitch, 1), shift).fill_(False)
        assert torch.equal(base[edge], before[edge])


@pytest.mark.parametrize("V", [1, 40, 257, 5000, 33000])
@pytest.mark.parametrize("dtype", [W.F32, W.BF16, W.F16])
def test_process_rows_on_odd_multiples_of_16_bytes(V, dtype):
    """Logits, results or both start 16 bytes past a 32-byte boundary."""
    size = 4 if dtype == W.F32 else 2
    for code in {dtype, W.F32}:
        osize = 4 if code == W.F32 else 2
        for x16, y16 in ((True, False), (False, True), (True, True)):
            p = Problem(17, 15, V, dtype, pitch=(-V) % 64, shift=16 // size if x16 else 0)
            ld = -(-V // 16) * 16
            buf = torch.full((15 * ld + 64,), 5.0, dtype=TYPES[code], device="cuda")
            out = torch.as_strided(buf, (15, V), (ld, 1), 16 // osize if y16 else 0)
            assert p.logits.data_ptr() % 32 == (16 if x16 else 0)
            assert out.data_ptr() % 32 == (16 if y16 else 0)
            gs.process_logits(p.logits, out=out, **p.kw)
            cu.check_values(out_values(out), *p.want(), code, "%s %s" % (x16, y16))
            rest = torch.ones_like(buf, dtype=torch.bool)
            torch.as_strided(rest, (15, V), (ld, 1), 16 // osize if y16 else 0).fill_(False)
            assert bool((buf[rest] == 5.0).all())
    p = Problem(18, 15, V, dtype, pitch=(-V) % 64, shift=16 // size)
    want = p.want()
    gs.process_logits(p.logits, out=p.logits, **p.kw)
    cu.check_values(out_values(p.logits), *want, dtype, "in place")


def test_process_allocates_rows_on_32_byte_boundaries():
    for V, dtype in ((33, torch.float32), (33, torch.float16), (64, torch.bfloat16)):
        y = gs.process_logits(torch.zeros(3, V, dtype=dtype, device="cuda"))
        assert y.shape == (3, V) and y.stride(1) == 1
        assert y.data_ptr() % 32 == 0 and y.stride(0) * y.element_size() % 32 == 0
        assert y.is_contiguous() == (V == 64)


def test_process_results_elsewhere_keep_their_surroundings():
    p = Problem(8, 12, 777, W.BF16)
    for ld, shift in ((777, 0), (784, 0), (800, 3), (1600, 777)):
        buf = torch.full((12 * ld + shift + 16,), 5.0, dtype=torch.float32, device="cuda")
        out = torch.as_strided(buf, (12, 777), (ld, 1), shift)
        gs.process_logits(p.logits, out=out, **p.kw)
        cu.check_values(out_values(out), *p.want(), W.F32)
        rest = torch.ones_like(buf, dtype=torch.bool)
        torch.as_strided(rest, (12, 777), (ld, 1), shift).fill_(False)
        assert bool((buf[rest] == 5.0).all())
    # the other half of the same buffer
    buf = torch.zeros(12, 1600, dtype=torch.bfloat16, device="cuda")
    buf[:, :777] = p.logits
    gs.process_logits(buf[:, :777], out=buf[:, 800:1577], **p.kw)
    cu.check_values(out_values(buf[:, 800:1577]), *p.want(), W.BF16)
    a, b = buf[:, :777].contiguous(), p.logits.contiguous()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_process_values_of_the_type_limits():
    """Biases and masks at the types' ends: sums that leave the range, the
    lowest value as an upstream mask, subnormals."""
    for dtype, low in ((W.F32, -3.4028235e38), (W.BF16, -3.3895314e38), (W.F16, -65504.0)):
        V = 64
        x = np.zeros((2, V), np.float32)
        x[:, 0::4], x[:, 1::4], x[:, 2::4] = low, -low, -np.inf
        x[:, 3::8] = W.roundtrip(np.full(8, 6e-8, np.float32), dtype)
        s = cu.HostState(2, V)
        s.set_bias(0, range(V), np.tile([-np.inf, np.inf, 1e38, -1e38, np.nan, 0, 1e-40, 3e38], 8))
        s.append(1, range(V), False)
        s.append(1, range(V), True)
        p = [np.float32([1.7, 1e30]), np.float32([0, 1e30]), np.float32([0, -1e30])]
        got = gs.process_logits(to_device(W.encode(x, dtype), dtype), state=upload(s),
                                repetition=dev(p[0]), frequency=dev(p[1]), presence=dev(p[2]),
                                out_dtype=torch.float32)
        h, b = s.history[:, :V], s.bias[:, :V]
        want = cu.binary32(W.roundtrip(x, dtype), h, b, *p, np.ones((2, V), bool))
        got = got.cpu().numpy()
        assert np.array_equal(got, want, equal_nan=True)


def test_bits_of_the_written_logits_are_the_formulas_in_binary32():
    p = Problem(9, 16, 3001, W.F32, tokens=400)
    got = gs.process_logits(p.logits, **p.kw).cpu().numpy()
    assert np.array_equal(got, cu.binary32(*p.parts()), equal_nan=True)


@pytest.mark.parametrize("dtype", [W.F32, W.BF16, W.F16])
@pytest.mark.parametrize("B", [3, 170])
def test_every_element_touched(dtype, B):
    """More touched elements than any list holds at a time: written, in place
    and drawn, on aligned and unaligned rows."""
    V = 5003
    for pitch, shift in (((-V) % 64, 0), (3, 1)):
        p = Problem(19, B, V, dtype, special=False, pitch=pitch, shift=shift)
        rng = np.random.default_rng(19)
        h = rng.integers(0, 4, p.host.history.shape).astype(np.uint32)
        h |= rng.integers(0, 2, h.shape).astype(np.uint32) << np.uint32(31)
        p.host.history[:], p.host.touched[:] = h, True
        p.host.history[:, V:] = 0
        p.host.bias[:, :V] = rng.uniform(-3, 3, (p.host.rows, V))
        p.kw["state"] = upload(p.host)
        got, want, _ = draw_both(p, rng)
        assert np.array_equal(got, want)
        code = dtype
        cu.check_values(out_values(gs.process_logits(p.logits, **p.kw)), *p.want(), code)
        want = p.want()
        gs.process_logits(p.logits, out=p.logits, **p.kw)
        cu.check_values(out_values(p.logits), *want, code)


# ---- the draw ---------------------------------------------------------------------
def keys(rng, B, greedy=0.25):
    T = rng.uniform(0.3, 2.0, B).astype(np.float32)
    T[rng.random(B) < greedy] = 0.0
    if B > 5:
        T[5] = np.nan
    seed = rng.integers(0, 1 << 63, B).astype(np.uint64)
    offset = rng.integers(0, 1 << 40, B).astype(np.uint64)
    return T, seed, offset


def draw_both(p, rng, **over):
    """The constrained draw, and the plain sampler on the written logits."""
    T, seed, offset = keys(rng, p.B)
    T = over.get("T", T)
    args = dev(T), gs.seeds_as_tensor(seed, "cuda"), gs.seeds_as_tensor(offset, "cuda")
    got = gs.constrained_gumbel_argmax(p.logits, *args, **p.kw)
    y = gs.process_logits(p.logits, out_dtype=torch.float32, **p.kw)
    want = gs.gumbel_argmax(y, *args)
    return got.cpu().numpy(), want.cpu().numpy(), (T, seed, offset)


@pytest.mark.parametrize("V", SIZES)
@pytest.mark.parametrize("dtype", [W.F32, W.BF16, W.F16])
def test_draw_equals_the_sampler_on_the_written_logits(V, dtype):
    rng = np.random.default_rng([V, dtype])
    for B, pitch, shift in ((1, 0, 0), (15, (-V) % 64, 0), (15, 3, 1), (70, (-V) % 64, 0),
                            (170, (-V) % 64, 0), (170, 3, 1)):
        for special in (False, True):
            p = Problem(10, B, V, dtype, special=special, pitch=pitch, shift=shift)
            got, want, _ = draw_both(p, rng)
            assert np.array_equal(got, want), (B, pitch, special,
                                               np.nonzero(got != want)[0][:5])


@pytest.mark.parametrize("state,mask", [(True, False), (False, True), (False, False)])
def test_draw_with_parts_absent(state, mask):
    rng = np.random.default_rng(11)
    for B in (3, 100, 200):
        for dtype in (W.F32, W.BF16):
            p = Problem(11, B, 5000, dtype, special=False, state=state, mask=mask)
            got, want, _ = draw_both(p, rng)
            assert np.array_equal(got, want)


def tally(t, got, y, T, ref, gap, where):
    """Rows with one finite candidate or none, or with +inf ones, have no near
    tie: they are compared exactly, and only the others go into the table."""
    n = (y > -np.inf).sum(1)
    plain = (n < 2) | (y == np.inf).any(1)
    assert np.array_equal(got[plain], ref[plain]), where
    t.add(got[~plain], ref[~plain], gap[~plain], ~(T > 0)[~plain], where)


@pytest.mark.parametrize("B,V,dtype", [(4, 32768, W.F32), (33, 20000, W.BF16),
                                       (300, 9001, W.F16), (130, 40000, W.BF16),
                                       (160, 40000, W.BF16)])
def test_draw_against_the_oracle(B, V, dtype):
    rng = np.random.default_rng([12, B])
    p = Problem(12, B, V, dtype, special=False, tokens=2000)
    got, _, (T, seed, offset) = draw_both(p, rng)
    y = cu.binary32(*p.parts())
    ref, gap = oracle.gumbel_argmax(y, T, seed, offset)
    t = Tally()
    tally(t, got, y, T, ref, gap, "B %d V %d" % (B, V))
    register("7 constrained draw", t, assert_bound=False)


@pytest.mark.parametrize("B", [2, 80, 200])
@pytest.mark.parametrize("dtype", [W.F32, W.BF16, W.F16])
def test_draw_rows_with_nothing_or_one_token_left(B, dtype):
    V = 6000
    rng = np.random.default_rng(13)
    x = logits_for(rng, B, V, dtype, special=False)
    bits = np.zeros((B, V), bool)
    only = rng.integers(0, V, B)
    only[0], only[1] = V - 1, 0
    bits[np.arange(B), only] = True
    bits[B // 2:] = False
    kw = dict(mask=dev(cu.pack_bits(bits)))
    T = np.where(np.arange(B) % 3 == 0, 0.0, 1.0).astype(np.float32)
    lg = to_device(W.encode(x, dtype), dtype)
    got = gs.constrained_gumbel_argmax(lg, dev(T), 5, 6, **kw).cpu().numpy()
    want = np.where(np.arange(B) < B // 2, only, -1)
    assert np.array_equal(got, want)
    # a NaN, +inf or masked token is no candidate where the mask forbids it; a NaN or -inf
    # token is none where it is the only one allowed
    for value, left in ((np.nan, -1), (-np.inf, -1), (np.inf, None)):
        y = x.copy()
        y[np.arange(B), only] = value
        y[:, 17] = np.inf
        lg = to_device(W.encode(W.roundtrip(y, dtype), dtype), dtype)
        got = gs.constrained_gumbel_argmax(lg, dev(T), 5, 6, **kw).cpu().numpy()
        w = np.where(np.arange(B) < B // 2, only if left is None else left, -1)
        w = np.where((only == 17) & (np.arange(B) < B // 2), 17, w)
        assert np.array_equal(got, w)


@pytest.mark.parametrize("B", [3, 90, 180])
@pytest.mark.parametrize("dtype", [W.BF16, W.F16, W.F32])
def test_draw_bans_and_forces_by_bias(B, dtype):
    V = 9000
    rng = np.random.default_rng(14)
    x = logits_for(rng, B, V, dtype, special=False)
    s = cu.HostState(B, V)
    forced = rng.integers(0, V, B)
    for r in range(B):
        if r % 3 == 0:
            s.set_bias(r, [forced[r]], [200.0])
        elif r % 3 == 1:
            s.set_bias(r, [forced[r]], [np.inf])
        else:
            s.set_bias(r, [int(x[r].argmax())], [-np.inf])
    p = Problem(14, B, V, dtype, special=False)
    p.logits = to_device(W.encode(x, dtype), dtype)
    p.kw = dict(state=upload(s))
    for greedy in (0.0, 1.0):
        T = np.full(B, 1.0 - greedy, np.float32)
        got, want, _ = draw_both(p, rng, T=T)
        assert np.array_equal(got, want)
        hit = np.arange(B) % 3 < 2
        assert np.array_equal(got[hit], forced[hit])
        assert (got[~hit] != x[~hit].argmax(1)).all()


@pytest.mark.parametrize("T", [1e-30, 1e-21, 1e-3, 50.0, 1e21, np.inf])
def test_draw_at_extreme_temperatures(T):
    rng = np.random.default_rng(15)
    for B in (4, 80, 160):
        for dtype in (W.F32, W.BF16):
            p = Problem(15, B, 3000, dtype, special=False, tokens=300)
            got, want, _ = draw_both(p, rng, T=np.full(B, T, np.float32))
            assert np.array_equal(got, want)


def test_draw_ties_go_to_the_lowest_index():
    """Equal constrained logits, some of them penalised down to the value of
    others, greedily: the lowest index."""
    V = 8000
    for B in (2, 70, 170):
        for dtype in (W.F32, W.BF16, W.F16):
            x = np.zeros((B, V), np.float32)
            s = cu.HostState(B, V)
            want = np.zeros(B, np.int64)
            for b in range(B):
                low = 3 + 41 * b
                x[b, low + 9], x[b, low], x[b, low + 5] = 2.0, 4.0, 2.0
                s.append(b, [low], False)  # 4 / 2 = 2, the lowest of three equal ones
                want[b] = low
            kw = dict(state=upload(s), repetition=2.0)
            lg = to_device(W.encode(x, dtype), dtype)
            got = gs.constrained_gumbel_argmax(lg, 0.0, 1, 2, **kw).cpu().numpy()
            assert np.array_equal(got, want)


def test_draw_frequencies_follow_the_constrained_softmax():
    """40 tokens, penalised, biased and masked: 2e5 draws a row against the
    softmax of the constrained logits (chi-square, 6 sigma)."""
    B, V, n = 4, 40, 200_000
    p = Problem(16, B, V, W.F32, special=False, tokens=25)
    p.slots, p.mask_rows = np.arange(B, dtype=np.int32), np.array([0, 4, -1, 0], np.int32)
    p.kw.update(slots=dev(p.slots), mask_rows=dev(p.mask_rows))
    y, _ = p.want()
    big = {k: (v.repeat(n // 1000) if k in ("slots", "repetition", "frequency", "presence",
                                           "mask_rows") else v) for k, v in p.kw.items()}
    lg = p.logits.repeat(n // 1000, 1)
    for k in ("slots", "repetition", "frequency", "presence", "mask_rows"):
        big[k] = p.kw[k].repeat(n // 1000)
    counts = np.zeros((B, V))
    for step in range(1000):
        seed = torch.arange(lg.shape[0], device="cuda", dtype=torch.int64)
        i = gs.constrained_gumbel_argmax(lg, 1.0, seed, step, **big).view(-1, B)
        counts += torch.stack([torch.bincount(i[:, b], minlength=V) for b in range(B)]) \
            .cpu().numpy()
    for b in range(B):
        e = np.exp(y[b] - y[b][np.isfinite(y[b])].max())
        q = e / e.sum()
        assert (counts[b][q == 0] == 0).all()
        keep = q * n > 10
        chi = ((counts[b] - n * q)[keep] ** 2 / (n * q)[keep]).sum()
        dof = keep.sum() - 1
        assert chi < dof + 6 * np.sqrt(2 * dof) + 6, (b, chi, dof)


# ---- as a server uses them ----------------------------------------------------------
def test_a_decode_loop():
    """Admission, then steps of draw and append; forked and finished requests
    in between. Every draw is the oracle's on the binary32 formula."""
    rng = np.random.default_rng(20)
    R, B, V = 12, 9, 4001
    s = cu.HostState(R, V)
    state = gs.new_logit_state(R, V)
    slots = rng.permutation(R)[:B].astype(np.int32)
    prompts, offsets = ragged(rng, rng.integers(0, 300, B), V)
    gs.history_append(state, dev(prompts), slots=dev(slots), offsets=dev(offsets), prompt=True)
    ids = rng.integers(0, V, (B, 5))
    vals = rng.uniform(-4, 4, (B, 5)).astype(np.float32)
    gs.bias_set(state, dev(ids.reshape(-1)), dev(vals.reshape(-1)), slots=dev(slots),
                offsets=dev(np.arange(B + 1) * 5))
    for i, r in enumerate(slots):
        s.append(r, prompts[offsets[i]:offsets[i + 1]], True)
        s.set_bias(r, ids[i], vals[i])
    rep, freq, pres = np.full(B, 1.3, np.float32), np.full(B, 0.4, np.float32), \
        np.full(B, 0.2, np.float32)
    T = np.where(np.arange(B) % 4 == 0, 0, 0.9).astype(np.float32)
    seed = W.splitmix64(7, B)
    ws = gs.new_workspace(B)
    seen = Tally()
    for step in range(12):
        if step == 5:  # request 0 is forked into a free slot's row; request 1 ends
            free = next(r for r in range(R) if r not in slots)
            for t in (state.history, state.bias, state.touched):
                t[free] = t[int(slots[0])]
            for a in (s.history, s.bias, s.touched):
                a[free] = a[slots[0]]
            gs.state_reset(state, slots=dev(slots[1:2]))
            s.reset(slots[1])
            slots[1] = free
        x = (rng.standard_normal((B, V)) * 3).astype(np.float32)
        bits = cu.random_mask(rng, B, V, ("free", "half", "few"))
        args = dev(x), dev(T), gs.seeds_as_tensor(seed, "cuda"), step
        got = gs.constrained_gumbel_argmax(*args, state=state, slots=dev(slots),
                                           repetition=dev(rep), frequency=dev(freq),
                                           presence=dev(pres), mask=dev(cu.pack_bits(bits)),
                                           workspace=ws)
        gs.history_append(state, got, slots=dev(slots))
        got = got.cpu().numpy()
        y = cu.binary32(x, s.history[slots, :V], s.bias[slots, :V], rep, freq, pres, bits)
        want, gap = oracle.gumbel_argmax(y, T, seed, np.full(B, step, np.uint64))
        tally(seen, got, y, T, want, gap, "step %d" % step)
        for i, r in enumerate(slots):
            s.append(r, [got[i]], False)
    same_state(state, s)
    register("7 constrained draw", seen, assert_bound=False)


def test_constrained_logits_feed_the_other_samplers():
    p = Problem(21, 20, 6000, W.F32, special=False)
    rng = np.random.default_rng(21)
    T, seed, offset = keys(rng, 20)
    args = dev(T), gs.seeds_as_tensor(seed, "cuda"), gs.seeds_as_tensor(offset, "cuda")
    y = gs.process_logits(p.logits, **p.kw)
    host = cu.binary32(*p.parts())
    got = gs.filtered_gumbel_argmax(y, *args, top_k=7).cpu().numpy()
    want, gap, edge = oracle.filtered_gumbel_argmax(host, T, seed, offset,
                                                    top_k=np.full(20, 7, np.int32))
    near = ((gap < 1e-5) | (edge < 1e-5)) & (T > 0)
    assert ((got == want) | near).all()
    assert np.array_equal(gs.argmax(y).cpu().numpy(), oracle.argmax(host)[0])


@pytest.mark.parametrize("B", [6, 100, 200])
def test_captured_and_replayed_on_another_stream(B):
    """A decode step (draw, append) captured once and replayed, as the eager
    steps on another copy of the state."""
    p = Problem(22, B, 3000, W.BF16, special=False)
    rng = np.random.default_rng(22)
    T, seed, _ = keys(rng, B)
    T, S = dev(T), gs.seeds_as_tensor(seed, "cuda")
    offset = torch.zeros(B, dtype=torch.int64, device="cuda")
    live = np.where((p.slots >= 0) & (p.slots < p.host.rows), p.slots, -1).astype(np.int32)

    def step(kw, out, ws):
        gs.constrained_gumbel_argmax(p.logits, T, S, offset, out=out, workspace=ws, **kw)
        gs.history_append(kw["state"], out, slots=kw["slots"])

    runs = []
    for captured in (False, True):
        kw = dict(p.kw, state=upload(p.host), slots=dev(live))
        out = torch.zeros(B, dtype=torch.int64, device="cuda")
        ws = gs.new_workspace(B)
        offset.zero_()
        seen = []
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            if captured:
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=side):
                    step(kw, out, ws)
            for i in range(6):
                offset.fill_(i)
                g.replay() if captured else step(kw, out, ws)
                seen.append(out.clone())
        torch.cuda.synchronize()
        runs.append((torch.stack(seen).cpu().numpy(), kw["state"].history.cpu().numpy(),
                     kw["state"].touched.cpu().numpy()))
    for a, b in zip(*runs):
        assert np.array_equal(a, b)


def test_two_streams_share_a_state_that_neither_writes():
    p = Problem(23, 180, 20000, W.BF16, special=False)
    T, seed, offset = keys(np.random.default_rng(23), 180)
    args = dev(T), gs.seeds_as_tensor(seed, "cuda"), gs.seeds_as_tensor(offset, "cuda")
    want = gs.constrained_gumbel_argmax(p.logits, *args, **p.kw)
    y = gs.process_logits(p.logits, **p.kw)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for st in streams:
        with torch.cuda.stream(st):
            ws = gs.new_workspace(180)
            for _ in range(5):
                got.append((gs.constrained_gumbel_argmax(p.logits, *args, workspace=ws, **p.kw),
                            gs.process_logits(p.logits, **p.kw)))
    torch.cuda.synchronize()
    for i, z in got:
        assert torch.equal(i, want)
        assert torch.equal(z.view(torch.int16), y.view(torch.int16))


def test_workspace_is_left_clean():
    p = Problem(24, 200, 3000, W.BF16)
    ws = gs.new_workspace(200)
    rng = np.random.default_rng(24)
    T, seed, offset = keys(rng, 200)
    args = dev(T), gs.seeds_as_tensor(seed, "cuda"), gs.seeds_as_tensor(offset, "cuda")
    a = gs.constrained_gumbel_argmax(p.logits, *args, workspace=ws, **p.kw)
    assert not bool(ws.any())
    b = gs.constrained_gumbel_argmax(p.logits, *args, workspace=ws, **p.kw)
    assert torch.equal(a, b)


def test_python_refusals():
    p = Problem(25, 8, 100, W.F32)
    st = p.kw["state"]
    x = p.logits
    for kw in (dict(slots=p.kw["slots"]), dict(repetition=1.2), dict(mask_rows=p.kw["mask_rows"]),
               dict(state=gs.new_logit_state(8, 101)), dict(state=gs.new_logit_state(7, 100)),
               dict(state=st, slots=p.kw["slots"].long()), dict(state=st, slots=p.kw["slots"][:4]),
               dict(state=st, frequency=torch.zeros(8)), dict(mask=p.kw["mask"].long()),
               dict(mask=p.kw["mask"][:, :3]), dict(mask=p.kw["mask"][:7]),
               dict(mask=p.kw["mask"].cpu()), dict(mask=p.kw["mask"][:1].expand(8, 4)),
               dict(mask=p.kw["mask"].repeat(1, 2)[:, ::2])):
        with pytest.raises(ValueError):
            gs.process_logits(x, **kw)
        with pytest.raises(ValueError):
            gs.constrained_gumbel_argmax(x, 1.0, 0, 0, **kw)
    for kw in (dict(out=x[:4]), dict(out=x.half()), dict(out_dtype=torch.bfloat16),
               dict(out=torch.empty_like(x), out_dtype=torch.float16),
               dict(out=torch.empty(100, 8, device="cuda").t())):
        with pytest.raises((ValueError, TypeError)):
            gs.process_logits(x, **kw)
    with pytest.raises(gs.GSampleError):
        big = torch.zeros(9, 100, device="cuda")
        gs.process_logits(big[:8], out=big[1:])  # rows shifted over each other
    tok = torch.zeros(8, dtype=torch.int64, device="cuda")
    one = torch.zeros(8, device="cuda")
    for call in (lambda: gs.history_append(st, tok.int()), lambda: gs.history_append(st, tok.cpu()),
                 lambda: gs.history_append(st, tok, slots=p.kw["slots"][:3]),
                 lambda: gs.history_append(st, tok, offsets=tok[:0]),
                 lambda: gs.bias_set(st, tok, one[:3]), lambda: gs.bias_set(st, tok, tok),
                 lambda: gs.bias_set(gs.new_logit_state(8, 9, bias=False), tok, one),
                 lambda: gs.state_reset(st, slots=tok),
                 lambda: gs.LogitState(st.history, st.bias, st.touched[:, :1], 100),
                 lambda: gs.LogitState(st.history[:, :100], st.bias, st.touched, 100),
                 lambda: gs.LogitState(st.history, st.bias.double(), st.touched, 100)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("B", [5, 90, 170])
def test_wider_states_and_masks(B):
    """State rows and mask rows with room to spare, mask words that start
    anywhere, and mask bits past the vocabulary set."""
    for V, dtype in ((77, W.F32), (1000, W.BF16), (6001, W.F16)):
        p = Problem(27, B, V, dtype, special=False)
        rng = np.random.default_rng([27, B])
        got, want, keys_ = draw_both(p, rng)
        written = gs.process_logits(p.logits, **p.kw)
        wide = cu.HostState(p.host.rows, V, ld=p.host.ld + 96)
        for a, b in ((wide.history, p.host.history), (wide.bias, p.host.bias),
                     (wide.touched, p.host.touched)):
            a[:, :V] = b[:, :V]
        words = cu.pack_bits(p.bits)
        n, w = words.shape
        if V % 32:
            words[:, -1] |= np.uint32((0xFFFFFFFF << (V % 32)) & 0xFFFFFFFF)
        buf = np.full(n * (w + 3) + 5, 0xFFFFFFFF, np.uint32)
        view = torch.as_strided(dev(buf), (n, w), (w + 3, 1), 1)
        view.copy_(dev(words))
        kw = dict(p.kw, state=upload(wide), mask=view)
        T, seed, offset = keys_
        again = gs.constrained_gumbel_argmax(p.logits, dev(T), gs.seeds_as_tensor(seed, "cuda"),
                                             gs.seeds_as_tensor(offset, "cuda"), **kw)
        assert np.array_equal(got, want) and np.array_equal(again.cpu().numpy(), want)
        assert torch.equal(gs.process_logits(p.logits, **kw), written)


def test_more_rows_than_a_grid_dimension():
    B, V = 70000, 37
    rng = np.random.default_rng(28)
    x = logits_for(rng, B, V, W.BF16, special=False)
    s = cu.HostState(B, V)
    t = rng.integers(0, V, (B, 2))
    rows = np.arange(B)
    s.history[rows, t[:, 0]] |= np.uint32(0x80000000)
    np.add.at(s.history, (rows, t[:, 1]), np.uint32(1))
    s.touched[rows, t[:, 0]] = s.touched[rows, t[:, 1]] = True
    state = gs.new_logit_state(B, V)
    gs.history_append(state, dev(t[:, 0]), prompt=True)
    gs.history_append(state, dev(t[:, 1]))
    same_state(state, s)
    bits = rng.random((B, V)) < 0.5
    kw = dict(state=state, repetition=1.5, frequency=0.5, mask=dev(cu.pack_bits(bits)))
    lg = to_device(W.encode(x, W.BF16), W.BF16)
    y = gs.process_logits(lg, out_dtype=torch.float32, **kw)
    one = np.ones(B)
    want = cu.constrained(x, s.history[:, :V], s.bias[:, :V], 1.5 * one, 0.5 * one, 0 * one, bits)
    cu.check_values(out_values(y), *want, W.F32)
    T = dev(np.where(rows % 3 == 0, 0, 1).astype(np.float32))
    a = gs.constrained_gumbel_argmax(lg, T, 3, 4, **kw)
    assert torch.equal(a, gs.gumbel_argmax(y, T, 3, 4))
    gs.state_reset(state)
    assert not bool(state.touched.any()) and not bool(state.history.any())


def test_empty_batches():
    x = torch.zeros(0, 50, device="cuda")
    assert gs.process_logits(x).shape == (0, 50)
    assert gs.constrained_gumbel_argmax(x, 1.0, 0, 0).shape == (0,)
    st = gs.new_logit_state(2, 50)
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    gs.history_append(st, none)
    gs.history_append(st, none, offsets=torch.zeros(3, dtype=torch.int64, device="cuda"))
    gs.bias_set(st, none, none.float())
    gs.state_reset(st, slots=none.int())
    assert not bool(st.touched.any())


# ---- positions past 32 bits -----------------------------------------------------------
def test_offsets_past_32_bits():
    """A state and a batch of more than 2^31 elements: the last rows."""
    V, R = 151936, 14400  # 2.19e9 elements
    if torch.cuda.mem_get_info()[0] < (60 << 30):
        pytest.skip("needs 60 GB of device memory")
    state = gs.new_logit_state(R, V)
    toks = torch.tensor([0, V - 1, V - 1, 5], device="cuda")
    slots = torch.tensor([R - 1, R - 1, R - 1, R - 2], dtype=torch.int32, device="cuda")
    gs.history_append(state, toks, slots=slots)
    gs.bias_set(state, toks[1:2], torch.tensor([3.0], device="cuda"), slots=slots[:1])
    assert state.history[R - 1, V - 1].item() == 2 and state.history[R - 1, 0].item() == 1
    assert state.history.count_nonzero().item() == 3
    x = torch.zeros(R, V, dtype=torch.bfloat16, device="cuda")
    x[R - 1, 77] = 1.5
    y = gs.process_logits(x, state=state, frequency=1.0)
    last = y[R - 1].float().cpu().numpy()
    want = np.zeros(V, np.float32)
    want[0], want[77], want[V - 1] = -1.0, 1.5, 1.0
    assert np.array_equal(last, want)
    assert y[R - 2, 5].item() == -1.0 and y[:R - 2].count_nonzero().item() == 0
    got = gs.constrained_gumbel_argmax(x, 0.0, 0, 0, state=state, frequency=1.0)
    assert got[R - 1].item() == 77 and not bool(got[:R - 1].any())
    # a forced token at the end of the last row, drawn
    gs.bias_set(state, toks[1:2], torch.tensor([500.0], device="cuda"), slots=slots[:1])
    got = gs.constrained_gumbel_argmax(x[R - 2:], 1.0, 0, 0, state=state, slots=slots[2:])
    assert got[0].item() == V - 1
    gs.state_reset(state, slots=slots[:1])
    assert state.history.count_nonzero().item() == 1 and state.bias.count_nonzero().item() == 0
